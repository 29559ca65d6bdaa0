"""Operators that train a model on the tokens its LM head sampled, for timing
and comparison: token log-probabilities of the head and their gradients, the
clipped policy loss, the preference loss, and global gradient-norm clipping.

``run`` makes one pass of a case, in plain torch (``own`` false: elementary
operations in fp32, fp64 where fp32 loses what matters) or through the
library (``own`` true).  ``exact`` is the same result from the definitions in
fp64.  Every random number is an input made by ``prepare``.
"""
import math
import random

import torch

own = False

# LM heads of this repository's workloads: (D, V, vocab_offset, vocabulary of
# the whole head).
HEADS = {
    "tiny": (256, 1000, 0, 1000),
    "llama3": (4096, 128256, 0, 128256),
    "qwen3": (5120, 151936, 0, 151936),
    "shard": (8192, 16032, 48096, 128256),
}


def _head(name, **kw):
    D, V, off, full = HEADS[name]
    return dict(D=D, V=V, offset=off, full=full, **kw)


def listed():
    return [
        # the log-probability a server returns with a single stream's token:
        # the decode step's own weights (fragment order), one row
        dict(name="logprob_decode_1", op="logprob", B=1, packed=True, temp="one", ignore=0.0,
             **_head("llama3")),
        # the same for a batch of streams with their own temperatures (some
        # greedy): also the old log-probabilities a rollout stores
        dict(name="logprob_decode_32", op="logprob", B=32, packed=True, temp="mixed", ignore=0.0,
             **_head("llama3")),
        # a training micro-batch of odd length on the longest vocabulary,
        # a quarter of its rows prompt tokens that carry no target
        dict(name="logprob_train_1777", op="logprob", B=1777, packed=False, temp="mixed",
             ignore=0.25, **_head("qwen3")),
        # a toy head: what a call costs when there is next to nothing to do
        dict(name="grad_tiny_4", op="grad", B=4, temp="one", ignore=0.0, **_head("tiny")),
        # one rank's vocabulary shard: most targets live on other ranks and
        # the log-sum-exp is the whole vocabulary's
        dict(name="grad_shard_513", op="grad", B=513, temp="one", ignore=0.25, **_head("shard")),
        # the ordinary training step of a 128k-row head
        dict(name="grad_train_4096", op="grad", B=4096, temp="one", ignore=0.25,
             **_head("llama3")),
        # a few short answers to one prompt, advantages per answer
        dict(name="policy_8", op="policy", S=8, mean_len=100, max_len=400, empty=0.0,
             per_token=False, ref=True, clip_low=0.2, clip_high=0.2, dual=0.0, kl_coef=0.05,
             kl="k3", reduction="token"),
        # a whole rollout batch with per-token advantages, prompts masked,
        # some answers masked out altogether
        dict(name="policy_512", op="policy", S=512, mean_len=1900, max_len=4096, empty=0.05,
             per_token=True, ref=True, clip_low=0.2, clip_high=0.28, dual=3.0, kl_coef=0.02,
             kl="k3", reduction="sequence"),
        # a small preference batch
        dict(name="preference_4", op="preference", P=4, mean_len=120, max_len=500, empty=0.0,
             ref=True, kind="sigmoid", beta=0.1, margin=0.0, smoothing=0.0, normalise=False),
        # long answers, label noise, some pairs padded away
        dict(name="preference_256", op="preference", P=256, mean_len=1900, max_len=4096,
             empty=0.05, ref=True, kind="sigmoid", beta=0.1, margin=0.0, smoothing=0.1,
             normalise=False),
        # adapters and norms of odd sizes, fp32, below the limit: nothing to scale
        dict(name="clip_adapters", op="clip", dtype="fp32", sizes="1,7,255,4096,4097,8192,12345,"
             "256,65536,1000,131,32768", rms=1e-4, max_norm=1.0),
        # a head and its model's matrices and norms in bf16, above the limit
        dict(name="clip_model", op="clip", dtype="bf16",
             sizes=f"{128256 * 4096},24x{4096 * 4096},33x4096", rms=1e-4, max_norm=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _sizes(text):
    """Tensor sizes of a clipping case: "count x size" or "size", in order."""
    out = []
    for part in text.split(","):
        count, _, size = part.rpartition("x")
        out += [int(size)] * int(count or 1)
    return out


def draw(rng):
    op = rng.choice(["logprob", "logprob", "grad", "grad", "policy", "preference", "clip"])
    if op in ("logprob", "grad"):
        limit = 4096 * 4096 * 128256 * (2 if op == "logprob" else 1)
        while True:
            D = 8 * _log_int(rng, 16, 1024)
            V = _log_int(rng, 500, 151936)
            B = _log_int(rng, 1, 8192)
            if B * D * V <= limit and D * V <= 151936 * 5120:
                break
        off = rng.choice([0, 0, rng.randrange(0, 100000)])
        c = dict(op=op, B=B, D=D, V=V, offset=off, full=off + V if off == 0 else off + 2 * V,
                 temp=rng.choice(["one", "mixed"]), ignore=rng.choice([0.0, 0.25, 0.6]))
        if op == "logprob":
            c["packed"] = False
            if rng.random() < 0.4:  # a decode head in fragment order (rows of a multiple of 32)
                c["packed"] = True
                c["D"] = max(64, D // 64 * 64)
        return c
    if op == "policy":
        return dict(op=op, S=_log_int(rng, 1, 512), mean_len=_log_int(rng, 4, 1900), max_len=4096,
                    empty=rng.choice([0.0, 0.1]), per_token=rng.random() < 0.5,
                    ref=rng.random() < 0.7, clip_low=rng.uniform(0.1, 0.3),
                    clip_high=rng.uniform(0.1, 0.4), dual=rng.choice([0.0, 3.0]),
                    kl_coef=rng.choice([0.0, 0.01, 0.1]), kl=rng.choice(["k1", "k2", "k3"]),
                    reduction=rng.choice(["token", "sequence"]))
    if op == "preference":
        kind = rng.choice(["sigmoid", "hinge", "ipo"])
        norm = rng.random() < 0.5
        return dict(op=op, P=_log_int(rng, 1, 256), mean_len=_log_int(rng, 4, 1900), max_len=4096,
                    empty=rng.choice([0.0, 0.1]), ref=rng.random() < 0.7, kind=kind,
                    beta=rng.uniform(1.0, 3.0) if norm else rng.uniform(0.05, 0.3),
                    margin=rng.choice([0.0, 0.5]) if kind != "ipo" else 0.0,
                    smoothing=rng.choice([0.0, 0.1]) if kind == "sigmoid" else 0.0,
                    normalise=norm)
    n = _log_int(rng, 1, 60)
    top = _log_int(rng, 1000, 200_000_000 // n)
    return dict(op="clip", dtype=rng.choice(["fp32", "bf16", "fp16"]),
                sizes=",".join(str(_log_int(rng, 1, top)) for _ in range(n)), rms=10 ** rng.uniform(-4.0, -2.0),
                max_norm=rng.choice([0.5, 1.0, 1e6]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _device():
    return torch.device("cuda")


def _inv_temperature(T):
    """fp32(1/T); a row whose temperature is not positive is scored unscaled."""
    pos = T > 0
    return torch.where(pos, 1.0 / torch.where(pos, T, torch.ones_like(T)), torch.ones_like(T))


def _prepare_head(case, g):
    dev = _device()
    B, D, V, off = case["B"], case["D"], case["V"], case["offset"]
    W = torch.empty(V, D, dtype=torch.bfloat16, device=dev)
    sigma = 1.28 / math.sqrt(D)  # logits of a model's head: standard deviation 1.28
    step = max(1, (1 << 26) // D)
    for r in range(0, V, step):
        n = min(step, V - r)
        W[r:r + n] = torch.randn(n, D, generator=g, device=dev) * sigma
    # targets in and outside this shard, some rows without one
    ids = torch.randint(0, case["full"], (B,), generator=g, device=dev)
    if case["full"] > off + V:  # half of a shard's targets are its own here
        mine = torch.rand(B, generator=g, device=dev) < 0.5
        ids = torch.where(mine, off + torch.randint(0, V, (B,), generator=g, device=dev), ids)
    # hidden states that favour the target by up to ~20 logits, RMS-normalised
    h = torch.randn(B, D, generator=g, device=dev)
    loc = (ids - off).clamp(0, V - 1)
    toward = W[loc].float()
    toward = toward / toward.norm(dim=1, keepdim=True) * math.sqrt(D)
    h = h + torch.rand(B, 1, generator=g, device=dev) * 0.25 * toward
    h = (h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + 1e-6)).to(torch.bfloat16)
    if case["temp"] == "one":
        T = torch.ones(B, device=dev)
    else:
        T = 0.3 + 1.2 * torch.rand(B, generator=g, device=dev)
        T[7::8] = 0.0
    ids = torch.where(torch.rand(B, generator=g, device=dev) < case["ignore"],
                      torch.full_like(ids, -100), ids).to(torch.int32)
    return dict(h=h, W=W, T=T, ids=ids)


def _forward(st, case, step=1024):
    """What the forward pass handed on: log-probability of each target and the
    log-sum-exp, over the whole vocabulary where W is one shard of it."""
    Wf = st["W"].float()
    inv_t = _inv_temperature(st["T"])
    loc = (st["ids"].long() - case["offset"])
    inside = (loc >= 0) & (loc < case["V"])
    lps, lses = [], []
    for r in range(0, st["h"].shape[0], step):
        z = ((st["h"][r:r + step].float() @ Wf.t()) * inv_t[r:r + step, None]).double()
        at = loc[r:r + step].clamp(0, case["V"] - 1)[:, None]
        zt = z.gather(1, at)[:, 0]
        own_t = inside[r:r + step]
        z.scatter_(1, at, torch.where(own_t, torch.full_like(zt, -math.inf), zt)[:, None])
        m = z.amax(dim=1).clamp(min=-1e300)
        rest = m + torch.log(torch.exp(z - m[:, None]).sum(dim=1))
        rest = rest + math.log(case["full"] / case["V"])  # other shards' share
        x = torch.where(own_t, rest - zt, rest)
        lp = -(torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs())))
        lses.append(torch.where(own_t, zt - lp, rest))
        lps.append(torch.where(own_t, lp, torch.full_like(lp, -12.0)))
    return torch.cat(lps).float(), torch.cat(lses).float()


def _lengths(n, mean, top):
    """Answer lengths as rollouts have them: log-normal, cut at the limit (the
    case's own set; `prepare` puts them in an order of the seed)."""
    rnd = random.Random(1000003 * n + mean)
    return [max(1, min(top, int(rnd.lognormvariate(math.log(mean) - 0.18, 0.6)))) for _ in range(n)]


def _prepare_sequences(case, n, seed, g):
    dev = _device()
    rnd = random.Random(seed)
    lens = _lengths(n, case["mean_len"], case["max_len"])
    rnd.shuffle(lens)
    cu, mask = [0], []
    for k in lens:
        cu.append(cu[-1] + k)
    N = cu[-1]
    prompt = [rnd.randrange(0, max(1, k // 3)) for k in lens]  # masked prefix
    cu_t = torch.tensor(cu, dtype=torch.int32, device=dev)
    gone = torch.tensor([1 if rnd.random() < case["empty"] else 0 for _ in range(n)], device=dev)
    seq = torch.bucketize(torch.arange(N, device=dev), cu_t[1:].long(), right=True)
    pos = torch.arange(N, device=dev) - cu_t[seq]
    mask = (pos >= torch.tensor(prompt, device=dev)[seq]) & (gone[seq] == 0)
    old = -2.0 * torch.empty(N, device=dev).exponential_(generator=g)
    return dict(cu=cu_t, mask=mask, old=old, N=N)


DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    st = dict(case=case)
    if op in ("logprob", "grad"):
        st.update(_prepare_head(case, g))
        if op == "grad":
            B = case["B"]
            st["lp"], st["lse"] = _forward(st, case)
            # what a policy loss hands back: advantages over the token count
            st["grad"] = torch.randn(B, generator=g, device=dev) / B
        elif case["packed"] and own:
            import lm_head_exact_amd as fs
            st["Wp"] = fs.pack_weights(st["W"], case["offset"])
    elif op == "policy":
        s = _prepare_sequences(case, case["S"], seed, g)
        N = s["N"]
        st.update(s)
        st["lp"] = s["old"] + 0.15 * torch.randn(N, generator=g, device=dev)
        st["ref"] = (s["old"] + 0.25 * torch.randn(N, generator=g, device=dev)
                     if case["ref"] else None)
        st["adv"] = torch.randn(N if case["per_token"] else case["S"], generator=g, device=dev)
    elif op == "preference":
        s = _prepare_sequences(case, 2 * case["P"], seed, g)
        N = s["N"]
        st.update(s)
        st["lp"] = s["old"]
        st["ref"] = (s["old"] + 0.2 * torch.randn(N, generator=g, device=dev)
                     if case["ref"] else None)
    else:
        dt = DTYPES[case["dtype"]]
        st["grads"] = [(torch.randn(n, generator=g, device=dev) * case["rms"]).to(dt)
                       for n in _sizes(case["sizes"])]
        st["out"] = [torch.empty_like(x) for x in st["grads"]]
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import lm_head_exact_amd as fs
    c = st["case"]
    op = c["op"]
    if op == "logprob":
        if c["packed"]:
            lp, lse = fs.token_logprobs(st["h"], st["Wp"], st["T"], st["ids"],
                                        vocab_offset=c["offset"], V=c["V"])
        else:
            lp, lse = fs.token_logprobs(st["h"], st["W"], st["T"], st["ids"],
                                        vocab_offset=c["offset"])
        return dict(logprob=lp, lse=lse)
    if op == "grad":
        dh, dW = fs.token_logprobs_backward(st["h"], st["W"], st["T"], st["ids"], st["lp"],
                                            st["lse"], st["grad"], vocab_offset=c["offset"])
        return dict(grad_h=dh, grad_W=dW)
    if op == "policy":
        stats, grad = fs.policy_loss(
            st["lp"], st["old"], st["adv"], st["cu"], ref_logprob=st["ref"], mask=st["mask"],
            per_token=c["per_token"], clip_low=c["clip_low"], clip_high=c["clip_high"],
            dual_clip=c["dual"], kl_coef=c["kl_coef"], kl=c["kl"], reduction=c["reduction"])
        return dict(stats=stats, grad=grad)
    if op == "preference":
        stats, rewards, grad = fs.preference_loss(
            st["lp"], st["cu"], ref_logprob=st["ref"], mask=st["mask"], kind=c["kind"],
            beta=c["beta"], margin=c["margin"], label_smoothing=c["smoothing"],
            length_normalised=c["normalise"])
        return dict(stats=stats, rewards=rewards, grad=grad)
    norm = fs.clip_grad_norm(st["grads"], c["max_norm"], out=st["out"])
    return dict(norm=norm, grads=st["out"])


def _run_plain(st):
    c = st["case"]
    op = c["op"]
    if op == "logprob":
        inv_t = _inv_temperature(st["T"])
        z = (st["h"].float() @ st["W"].float().t()) * inv_t[:, None]
        m = z.amax(dim=1)
        lse = m + torch.log(torch.exp(z - m[:, None]).sum(dim=1))
        loc = st["ids"].long() - c["offset"]
        inside = (loc >= 0) & (loc < c["V"])
        # z_t - lse cancels for a likely target: with L the log-sum-exp of the
        # other ids it is -log(1 + exp(L - z_t))
        at = loc.clamp(0, c["V"] - 1)[:, None]
        zt = z.gather(1, at)[:, 0]
        z.scatter_(1, at, -math.inf)
        m = z.amax(dim=1).clamp(min=-3e38)
        x = m + torch.log(torch.exp(z - m[:, None]).sum(dim=1)) - zt
        lp = -(torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs())))
        lp = torch.where(inside, lp, torch.full_like(lse, -math.inf))
        lp = torch.where(st["ids"] < 0, torch.zeros_like(lp), lp)
        return dict(logprob=lp, lse=lse)
    if op == "grad":
        inv_t = _inv_temperature(st["T"])
        Wf, hf = st["W"].float(), st["h"].float()
        gr = torch.where(st["ids"] < 0, torch.zeros_like(st["grad"]), st["grad"])
        p = torch.exp((hf @ Wf.t()) * inv_t[:, None] - st["lse"][:, None])
        loc = st["ids"].long() - c["offset"]
        inside = (loc >= 0) & (loc < c["V"])
        rows = torch.arange(c["B"], device=p.device)[inside]
        dz = -p
        dz[rows, loc[inside]] = -torch.expm1(st["lp"][inside])
        dz = dz * (gr * inv_t)[:, None]
        return dict(grad_h=(dz @ Wf).to(torch.bfloat16), grad_W=(dz.t() @ hf).to(torch.bfloat16))
    if op == "policy":
        return _policy(st, torch.float32)
    if op == "preference":
        return _preference(st, torch.float32)
    total = torch.zeros((), dtype=torch.float64, device=_device())
    for x in st["grads"]:
        total = total + (x.float() * x.float()).sum(dtype=torch.float64)
    norm = torch.sqrt(total)
    coef = torch.clamp(c["max_norm"] / (norm + 1e-6), max=1.0).float()
    coef = torch.where(torch.isfinite(norm), coef, torch.ones_like(coef))
    for x, y in zip(st["grads"], st["out"]):
        y.copy_(x.float() * coef)
    return dict(norm=norm.float().reshape(1), grads=st["out"])


def _segments(st, n):
    cu = st["cu"].long()
    return torch.bucketize(torch.arange(st["N"], device=cu.device), cu[1:], right=True)


def _policy(st, work):
    """The clipped surrogate with a KL penalty; differences of log-probabilities
    and clipping borders in fp64 (a ratio next to a border decides whether a
    token has a gradient), the rest in `work` precision."""
    c = st["case"]
    S, dev = c["S"], st["lp"].device
    seq = _segments(st, S)
    m = st["mask"]
    d = st["lp"].double() - st["old"].double()
    A = st["adv"] if c["per_token"] else st["adv"][seq]
    pos, neg = A > 0, A < 0
    high = d > math.log1p(c["clip_high"])
    low = d < math.log1p(-c["clip_low"])
    r = torch.exp(d.to(work))
    A = A.to(work)
    rc = torch.where(high, torch.full_like(r, 1 + c["clip_high"]),
                     torch.where(low, torch.full_like(r, 1 - c["clip_low"]), r))
    clipped = (pos & high) | (neg & low)
    surr = -torch.where(clipped, rc, r) * A
    gs = torch.where(clipped, torch.zeros_like(r), -r * A)
    if c["dual"] > 0:
        cap = neg & (d > math.log(c["dual"]))
        surr = torch.where(cap, -c["dual"] * A, surr)
        gs = torch.where(cap, torch.zeros_like(gs), gs)
        clipped = clipped | cap
    kl, gk = torch.zeros_like(r), torch.zeros_like(r)
    if st["ref"] is not None:
        e64 = st["ref"].double() - st["lp"].double()
        e = e64.to(work)
        if c["kl"] == "k1":
            kl, gk = -e, torch.ones_like(e)
        elif c["kl"] == "k2":
            kl, gk = 0.5 * e * e, -e
        else:
            x = torch.expm1(e64)
            kl, gk = (x - e64).to(work), (-x).to(work)
    count = torch.zeros(S, dtype=torch.float64, device=dev).index_add_(0, seq, m.double())
    if c["reduction"] == "token":
        w = torch.ones(S, dtype=torch.float64, device=dev) / count.sum().clamp(min=1)
    else:
        w = 1.0 / (count.clamp(min=1) * (count > 0).sum().clamp(min=1))
    w = torch.where(m, w[seq], torch.zeros_like(d))
    zero = torch.zeros_like(d)
    surr_mean = (torch.where(m, surr.double(), zero) * w).sum()
    kl_mean = (torch.where(m, kl.double(), zero) * w).sum()
    frac = (clipped & m).sum().double() / m.sum().clamp(min=1).double()
    loss = surr_mean + c["kl_coef"] * kl_mean
    grad = torch.where(m, (gs + c["kl_coef"] * gk).double() * w, zero)
    out = torch.float32 if work is torch.float32 else torch.float64
    return dict(stats=torch.stack([loss, surr_mean, kl_mean, frac]).to(out), grad=grad.to(out))


def _preference(st, work):
    """Paired answers 0..P-1 (chosen) and P..2P-1 (rejected); sums over a
    sequence and their differences in fp64 (long sums, then cancellation)."""
    c = st["case"]
    P, dev = c["P"], st["lp"].device
    seq = _segments(st, 2 * P)
    m = st["mask"]
    d = st["lp"].double()
    if st["ref"] is not None:
        d = d - st["ref"].double()
    zeros = torch.zeros(2 * P, dtype=torch.float64, device=dev)
    s = zeros.index_add(0, seq, torch.where(m, d, torch.zeros_like(d)))
    n = zeros.index_add(0, seq, m.double())
    per = 1.0 / n.clamp(min=1) if c["normalise"] else torch.ones_like(n)
    s = s * per
    both = (n[:P] > 0) & (n[P:] > 0)
    pairs = both.sum().clamp(min=1).double()
    diff = s[:P] - s[P:]
    beta, eps = c["beta"], c["smoothing"]
    if c["kind"] == "ipo":
        t = diff - 1.0 / (2.0 * beta)
        loss, dl = t * t, 2.0 * t
    else:
        x = beta * diff - c["margin"]
        if c["kind"] == "hinge":
            loss, dl = torch.clamp(1.0 - x, min=0.0), torch.where(x < 1.0, -beta, 0.0).double()
        else:
            def softplus(v):
                return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-v.abs()))
            loss = (1 - eps) * softplus(-x) + eps * softplus(x)
            dl = beta * (eps - 1.0 / (1.0 + torch.exp(x)))
    loss = torch.where(both, loss, torch.zeros_like(loss)).sum() / pairs
    dl = torch.where(both, dl, torch.zeros_like(dl)) / pairs
    acc = ((diff > 0) & both).sum().double() / pairs
    gap = torch.where(both, beta * diff, torch.zeros_like(diff)).sum() / pairs
    grad = torch.where(m, (torch.cat([dl, -dl]) * per)[seq], torch.zeros_like(d))
    out = torch.float32 if work is torch.float32 else torch.float64
    return dict(stats=torch.stack([loss, acc, gap]).to(out), rewards=(beta * s).to(out),
                grad=grad.to(out))


def work(case):
    op = case["op"]
    if op in ("logprob", "grad"):
        B, D, V = case["B"], case["D"], case["V"]
        if op == "logprob":
            return {"bytes": 2 * V * D + 2 * B * D + 16 * B, "flops": 2 * B * V * D}
        return {"bytes": 4 * V * D + 4 * B * D + 20 * B, "flops": 6 * B * V * D}
    if op in ("policy", "preference"):
        n = case["S"] if op == "policy" else 2 * case["P"]
        N = sum(_lengths(n, case["mean_len"], case["max_len"]))
        if op == "policy":
            per = 4 * (3 + case["ref"] + case["per_token"]) + 1
        else:
            per = 4 * (2 + case["ref"]) + 1
        return {"bytes": per * N + 8 * n, "flops": (40 if op == "policy" else 4) * N}
    size = {"fp32": 4, "bf16": 2, "fp16": 2}[case["dtype"]]
    N = sum(_sizes(case["sizes"]))
    return {"bytes": 2 * size * N, "flops": 3 * N}


# ---------------------------------------------------------------------------
# the definitions in fp64, one sequence, tensor or block of rows at a time
# ---------------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False  # the inputs alone: no weights laid out for the library
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op in ("logprob", "grad"):
        return _exact_head(case, st)
    if op == "policy":
        return _exact_policy(case, st)
    if op == "preference":
        return _exact_preference(case, st)
    sq = sum((x.double() ** 2).sum().item() for x in st["grads"])
    norm = math.sqrt(sq)
    coef = min(1.0, case["max_norm"] / (norm + 1e-6))
    return dict(norm=torch.tensor([norm], dtype=torch.float64),
                grads=[x.double() * coef for x in st["grads"]])


def _exact_head(case, st):
    off, V, B = case["offset"], case["V"], case["B"]
    h, W = st["h"].double(), st["W"].double()
    beta = [1.0 / 1.0 if not t > 0 else float(torch.tensor(1.0) / torch.tensor(t)) for t in
            st["T"].tolist()]
    beta = torch.tensor(beta, dtype=torch.float64, device=h.device)
    ids = st["ids"].tolist()
    lps, lses = [], []
    gh, gw = torch.empty_like(h), torch.zeros_like(W)
    step = max(1, (1 << 27) // V)
    for r in range(0, B, step):
        e = min(B, r + step)
        z = torch.matmul(h[r:e], W.transpose(0, 1)) * beta[r:e].unsqueeze(1)
        if case["op"] == "logprob":
            l = torch.logsumexp(z, dim=1)
            lses.append(l)
            one = []
            for i in range(r, e):
                t = ids[i]
                if t < 0:
                    one.append(torch.zeros_like(l[0]))
                elif off <= t < off + V:
                    others = z[i - r].clone()
                    others[t - off] = -math.inf
                    one.append(-torch.logaddexp(torch.logsumexp(others, dim=0) - z[i - r, t - off],
                                                torch.zeros_like(l[0])))
                else:
                    one.append(torch.full_like(l[0], -math.inf))
            lps.append(torch.stack(one))
            continue
        dz = torch.exp(z - st["lse"][r:e].double().unsqueeze(1)).neg_()
        for i in range(r, e):
            if ids[i] < 0:
                dz[i - r] = 0.0
            elif off <= ids[i] < off + V:
                dz[i - r, ids[i] - off] = -torch.expm1(st["lp"][i].double())
        dz *= (st["grad"][r:e].double() * beta[r:e]).unsqueeze(1)
        gh[r:e] = torch.matmul(dz, W)
        gw += torch.matmul(dz.transpose(0, 1), h[r:e])
    if case["op"] == "logprob":
        return dict(logprob=torch.cat(lps), lse=torch.cat(lses))
    return dict(grad_h=gh, grad_W=gw)


def _exact_policy(case, st):
    cu = st["cu"].tolist()
    S, N = case["S"], st["N"]
    f64 = torch.float64
    lo, hi = 1 - case["clip_low"], 1 + case["clip_high"]
    mask = st["mask"].cpu()
    lp, old, adv = (st[k].double().cpu() for k in ("lp", "old", "adv"))
    ref = st["ref"].double().cpu() if st["ref"] is not None else None
    counts = [int(mask[cu[s]:cu[s + 1]].sum()) for s in range(S)]
    total, filled = max(1, sum(counts)), max(1, sum(1 for k in counts if k))
    grad = torch.zeros(N, dtype=f64)
    surr_sum = kl_sum = hit = 0.0
    for s in range(S):
        if counts[s] == 0:
            continue
        w = 1.0 / total if case["reduction"] == "token" else 1.0 / (counts[s] * filled)
        a, b = cu[s], cu[s + 1]
        keep = mask[a:b].nonzero()[:, 0] + a
        x = lp[keep]
        A = adv[keep] if case["per_token"] else adv[s].expand(len(keep))
        r = (x - old[keep]).exp()
        plain, bounded = r * A, r.clamp(lo, hi) * A
        take = torch.minimum(plain, bounded)
        live = plain <= bounded
        if case["dual"] > 0:
            floor = case["dual"] * A
            under = (A < 0) & (take < floor)
            take = torch.where(under, floor, take)
            live = live & ~under
        g = torch.where(live, -plain, torch.zeros_like(r))
        hit += float((~live).sum())
        surr_sum -= w * float(take.sum())
        if ref is not None:
            q = ref[keep] - x
            if case["kl"] == "k1":
                k, gk = -q, torch.ones_like(q)
            elif case["kl"] == "k2":
                k, gk = q * q / 2, -q
            else:
                k, gk = torch.expm1(q) - q, -torch.expm1(q)
            kl_sum += w * float(k.sum())
            g = g + case["kl_coef"] * gk
        grad[keep] = w * g
    stats = [surr_sum + case["kl_coef"] * kl_sum, surr_sum, kl_sum, hit / total]
    return dict(stats=torch.tensor(stats, dtype=f64), grad=grad)


def _exact_preference(case, st):
    cu = st["cu"].tolist()
    P, N = case["P"], st["N"]
    f64 = torch.float64
    mask = st["mask"].cpu()
    lp = st["lp"].double().cpu()
    x = lp - st["ref"].double().cpu() if st["ref"] is not None else lp
    keep = [mask[cu[s]:cu[s + 1]].nonzero()[:, 0] + cu[s] for s in range(2 * P)]
    score = []
    for k in keep:
        v = math.fsum(x[k].tolist())
        score.append(v / max(1, len(k)) if case["normalise"] else v)
    live = [p for p in range(P) if len(keep[p]) and len(keep[P + p])]
    n = max(1, len(live))
    beta, eps = case["beta"], case["smoothing"]

    def log_sigmoid(v):
        return min(v, 0.0) - math.log1p(math.exp(-abs(v)))

    def sigmoid(v):
        return math.exp(log_sigmoid(v))

    grad = torch.zeros(N, dtype=f64)
    loss = acc = gap = 0.0
    for p in live:
        d = score[p] - score[P + p]
        if case["kind"] == "ipo":
            one, g = (d - 0.5 / beta) ** 2, 2 * (d - 0.5 / beta)
        elif case["kind"] == "hinge":
            u = beta * d - case["margin"]
            one, g = max(0.0, 1 - u), -beta if u < 1 else 0.0
        else:
            u = beta * d - case["margin"]
            one = -(1 - eps) * log_sigmoid(u) - eps * log_sigmoid(-u)
            g = beta * (-(1 - eps) * sigmoid(-u) + eps * sigmoid(u))
        loss, acc, gap = loss + one / n, acc + (d > 0) / n, gap + beta * d / n
        for k, sign in ((keep[p], 1.0), (keep[P + p], -1.0)):
            grad[k] = sign * g / n / (len(k) if case["normalise"] else 1)
    return dict(stats=torch.tensor([loss, acc, gap], dtype=f64),
                rewards=torch.tensor([beta * v for v in score], dtype=f64), grad=grad)
