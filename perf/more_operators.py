"""Operators of the LM head beyond the bf16 samplers and log-probabilities, for
timing and comparison: the head in 8-bit floating point with a scale for each
block of 128 (quantising the weights, logits, samples and log-probabilities)
and the softmax cross entropy of the head with its gradients, without logits in
memory.

``run`` makes one pass of a case, in plain torch (``own`` false: elementary
operations in fp32, fp64 where fp32 loses what matters) or through the library
(``own`` true).  ``exact`` is the same result from the definitions in fp64.
Every random number is an input made by ``prepare``, or the counter-based noise
of the case's seed and step.

The 8-bit head.  A block's scale is the power of two 2^e with the least e
(-110 or more) for which no finite entry exceeds 448 * 2^e (e = 0 for a block of
zeros); its values are e4m3, rounded to nearest even.  Weights have blocks of
128 rows by 128 columns, hidden states of one row by 128 columns.
"""
import math

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
BLOCK = 128


def _head(name, **kw):
    D, V, off, full = HEADS[name]
    return dict(D=D, V=V, offset=off, full=full, **kw)


def listed():
    return [
        # a toy head in 8 bits, row-major as a checkpoint stores it: next to no work
        dict(name="quantize_tiny", op="quantize", packed=False, **_head("tiny")),
        # what a trainer does after every update for the rollouts that follow: the
        # whole head in the order that the decode step reads
        dict(name="quantize_rollout", op="quantize", packed=True, **_head("llama3")),
        # one stream's decode step whose logits a host-side constraint still edits
        dict(name="logits_decode_1", op="logits", B=1, dtype="fp32", **_head("llama3")),
        # logits of an odd number of positions on one rank's vocabulary shard
        dict(name="logits_shard_777", op="logits", B=777, dtype="bf16", **_head("shard")),
        # a decode step of a toy head: what a call costs
        dict(name="sample_tiny_4", op="sample", B=4, temp="one", **_head("tiny")),
        # the decode step of a batch of streams with their own temperatures (some greedy)
        dict(name="sample_decode_32", op="sample", B=32, temp="mixed", **_head("llama3")),
        # log-probabilities stored with a rollout's tokens, under the 8-bit policy that drew them
        dict(name="logprob_decode_32", op="logprob", B=32, temp="mixed", ignore=0.0,
             **_head("llama3")),
        # scoring an odd number of tokens with the 8-bit head, a quarter of them prompts
        dict(name="logprob_score_1777", op="logprob", B=1777, temp="one", ignore=0.25,
             **_head("qwen3")),
        # a toy head's training step
        dict(name="xent_tiny_4", op="xent", B=4, ignore=0.0, smoothing=0.0, z_loss=0.0,
             reduction="mean", grads=True, **_head("tiny")),
        # a small vocabulary, wide rows, smoothed labels and a penalty on the log-sum-exp
        dict(name="xent_smooth_513", op="xent", B=513, ignore=0.25, smoothing=0.1, z_loss=1e-4,
             reduction="sum", grads=True, **_head("shard")),
        # validation: the loss alone
        dict(name="xent_eval_1777", op="xent", B=1777, ignore=0.25, smoothing=0.0, z_loss=0.0,
             reduction="mean", grads=False, **_head("qwen3")),
        # the ordinary training step of a 128k-row head
        dict(name="xent_train_4096", op="xent", B=4096, ignore=0.25, smoothing=0.0, z_loss=1e-4,
             reduction="mean", grads=True, **_head("llama3")),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "logits", "logits", "sample", "logprob", "logprob", "xent", "xent",
                     "xent"])
    limit = 4096 * 4096 * 128256
    while True:
        D = 64 * _log_int(rng, 2, 128)
        V = _log_int(rng, 500, 151936)
        B = _log_int(rng, 1, 8192)
        if D * V <= 151936 * 5120 and B * D * V <= limit and B * V <= 4096 * 128256:
            break
    off = 4 * rng.choice([0, 0, rng.randrange(0, 25000)])
    c = dict(op=op, D=D, V=V, offset=off, full=V if off == 0 else off + 2 * V)
    if op == "quantize":
        return dict(c, packed=rng.random() < 0.6)
    if op == "logits":  # single steps in fp32, batches of positions in bf16
        return dict(c, B=B, dtype="fp32" if B <= 16 else "bf16")
    if op == "sample":
        return dict(c, B=_log_int(rng, 1, 32), temp=rng.choice(["one", "mixed"]))
    if op == "logprob":
        return dict(c, B=B, temp=rng.choice(["one", "mixed"]), ignore=rng.choice([0.0, 0.25, 0.6]))
    c["D"] = D - 8 * rng.randrange(0, 4)  # (the bf16 head takes any multiple of 8)
    return dict(c, B=B, offset=0, full=V, ignore=rng.choice([0.0, 0.25, 0.6]),
                smoothing=rng.choice([0.0, 0.0, 0.1]), z_loss=rng.choice([0.0, 1e-4, 1e-2]),
                reduction=rng.choice(["mean", "mean", "sum"]), grads=rng.random() < 0.75)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _weights(V, D, g):
    dev = g.device
    W = torch.empty(V, D, dtype=torch.bfloat16, device=dev)
    sigma = 1.28 / math.sqrt(D)  # logits of a model's head: standard deviation 1.28
    step = max(1, (1 << 26) // D)
    for r in range(0, V, step):
        n = min(step, V - r)
        W[r:r + n] = torch.randn(n, D, generator=g, device=dev) * sigma
    return W


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op, V, D, off = case["op"], case["V"], case["D"], case["offset"]
    st = dict(case=case, W=_weights(V, D, g))
    if op == "quantize":
        return st
    B = case["B"]
    # targets in and outside this shard
    ids = torch.randint(0, case["full"], (B,), generator=g, device=dev)
    if case["full"] > off + V and op != "xent":  # half of a shard's targets are its own here
        mine = torch.rand(B, generator=g, device=dev) < 0.5
        ids = torch.where(mine, off + torch.randint(0, V, (B,), generator=g, device=dev), ids)
    if op == "xent":
        ids = ids % V
        off = 0
    # hidden states that favour the target by up to ~20 logits, RMS-normalised
    h = torch.randn(B, D, generator=g, device=dev)
    toward = st["W"][(ids - off).clamp(0, V - 1)].float()
    toward = toward / toward.norm(dim=1, keepdim=True) * math.sqrt(D)
    h = h + torch.rand(B, 1, generator=g, device=dev) * 0.25 * toward
    st["h"] = (h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + 1e-6)).to(torch.bfloat16)
    if "temp" in case:
        T = torch.ones(B, device=dev)
        if case["temp"] == "mixed":
            T = 0.3 + 1.2 * torch.rand(B, generator=g, device=dev)
            T[7::8] = 0.0
        st["T"] = T
    if "ignore" in case:
        gone = torch.rand(B, generator=g, device=dev) < case["ignore"]
        st["ids"] = torch.where(gone, torch.full_like(ids, -100), ids).to(torch.int32)
    st["seed"], st["step"] = 1000 + seed, seed % 977
    if op in ("logits", "sample", "logprob"):
        # the head in 8 bits, as a server keeps it from its loading on
        if own:
            import lm_head_exact_amd as fs
            st["Wq"], st["scale"] = fs.quantize_weights_fp8(st["W"])
        else:
            st["Wq"], st["scale"] = _quantize(st["W"], BLOCK)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import lm_head_exact_amd as fs
    c = st["case"]
    op = c["op"]
    if op == "quantize":
        q, scale = fs.quantize_weights_fp8(st["W"], packed=c["packed"])
        return dict(q=q, scale=scale)
    if op == "logits":
        return dict(logits=fs.logits_fp8(st["h"], st["Wq"], st["scale"], c["V"],
                                         dtype=DTYPES[c["dtype"]]))
    if op == "sample":
        ids, val = fs.sample_fp8(st["h"], st["Wq"], st["scale"], c["V"], st["T"], st["seed"],
                                 st["step"], vocab_offset=c["offset"])
        return dict(ids=ids, maxval=val)
    if op == "logprob":
        lp, lse = fs.token_logprobs_fp8(st["h"], st["Wq"], st["scale"], c["V"], st["T"], st["ids"],
                                        vocab_offset=c["offset"])
        return dict(logprob=lp, lse=lse)
    stats, losses, gh, gw = fs.cross_entropy(
        st["h"], st["W"], st["ids"], label_smoothing=c["smoothing"], z_loss=c["z_loss"],
        reduction=c["reduction"], need_h=c["grads"], need_W=c["grads"])
    out = dict(stats=stats, losses=losses)
    return dict(out, grad_h=gh, grad_W=gw) if c["grads"] else out


def _blocks(x, rows):
    """x in blocks of `rows` by 128, padded by zeros."""
    R, D = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -D % BLOCK, 0, -R % rows))
    return x.view(x.shape[0] // rows, rows, x.shape[1] // BLOCK, BLOCK)


def _quantize(x, rows):
    """(e4m3 values, the blocks' scales) of x."""
    R, D = x.shape
    b = _blocks(x, rows)
    size = b.abs()
    amax = torch.where(torch.isfinite(size), size, torch.zeros_like(size)).amax(dim=(1, 3))
    m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-110)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    down = torch.ldexp(torch.ones_like(amax), -e)
    q = (b * down[:, None, :, None]).view(b.shape[0] * rows, -1)[:R, :D]
    return (q.to(torch.float8_e4m3fn),
            torch.ldexp(torch.ones_like(amax), e).to(torch.float8_e8m0fnu))


def _dequantize(q, scale, rows):
    R, D = q.shape
    b = _blocks(q, rows) * scale.float()[:, None, :, None]
    return b.view(b.shape[0] * rows, -1)[:R, :D]


def _logits(st):
    hq, hs = _quantize(st["h"], 1)
    return _dequantize(hq, hs, 1) @ _dequantize(st["Wq"], st["scale"], BLOCK).t()


def _inv_temperature(T):
    """fp32(1/T); a row whose temperature is not positive is scored unscaled."""
    pos = T > 0
    return torch.where(pos, 1.0 / torch.where(pos, T, torch.ones_like(T)), torch.ones_like(T))


def _noise(B, V, offset, seed, step, device):
    """Standard Gumbel noise of every row and global id: Philox-4x32-10 with
    counter (id / 4, row, step), key seed, word id mod 4, u = (x + 1/2) 2^-32."""
    low = 0xFFFFFFFF
    c0 = (offset // 4 + torch.arange((V + 3) // 4, device=device))[None, :].expand(B, -1)
    c1 = torch.arange(B, device=device)[:, None].expand_as(c0)
    c2, c3 = torch.full_like(c0, step & low), torch.full_like(c0, step >> 32)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        p, q = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((q >> 32) & low) ^ c1 ^ k0, q & low, ((p >> 32) & low) ^ c3 ^ k1, p & low)
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    x = torch.stack([c0, c1, c2, c3], dim=2).view(B, -1)[:, :V]
    return -torch.log(-torch.log((x.double() + 0.5) * 2.0 ** -32))


def _run_plain(st):
    c = st["case"]
    op = c["op"]
    if op == "quantize":
        q, scale = _quantize(st["W"], BLOCK)
        if c["packed"]:  # groups of 16 rows, 64 columns at a time, 16 bytes per row and quarter
            V, D = c["V"], c["D"]
            q = torch.cat([q.view(torch.uint8),
                           torch.zeros(-V % 16, D, dtype=torch.uint8, device=q.device)])
            q = q.view(-1, 16, D // 64, 4, 16).permute(0, 2, 3, 1, 4).reshape(-1)
            q = q.view(torch.float8_e4m3fn)
        return dict(q=q, scale=scale)
    if op == "xent":
        return _xent(st)
    z = _logits(st)
    if op == "logits":
        return dict(logits=z.to(DTYPES[c["dtype"]]))
    inv_t = _inv_temperature(st["T"])
    if op == "sample":
        s = z * inv_t[:, None]
        g = _noise(c["B"], c["V"], c["offset"], st["seed"], st["step"], z.device).float()
        s = torch.where((st["T"] > 0)[:, None], s + g, z)
        val, at = s.max(dim=1)
        return dict(ids=(at + c["offset"]).to(torch.int32), maxval=val)
    z = z * inv_t[:, None]
    m = z.amax(dim=1)
    lse = m + torch.log(torch.exp(z - m[:, None]).sum(dim=1))
    loc = st["ids"].long() - c["offset"]
    inside = (loc >= 0) & (loc < c["V"])
    lp = torch.where(inside, _of_target(z, loc.clamp(0, c["V"] - 1)), torch.full_like(lse, -math.inf))
    return dict(logprob=torch.where(st["ids"] < 0, torch.zeros_like(lp), lp), lse=lse)


def _of_target(z, at):
    """Log-probability of column `at` of each row of logits: z_t - logsumexp
    cancels for a likely target; with L the log-sum-exp of the others it is
    -log(1 + exp(L - z_t)).  Overwrites z."""
    zt = z.gather(1, at[:, None])[:, 0]
    z.scatter_(1, at[:, None], -math.inf)
    m = z.amax(dim=1).clamp(min=-3e38)
    x = m + torch.log(torch.exp(z - m[:, None]).sum(dim=1)) - zt
    return -(torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs())))


def _xent(st):
    """Mean or sum over the rows with a target of
    (1 - s) (lse - z_y) + s (lse - mean z) + z_loss lse^2."""
    c = st["case"]
    V, eps = c["V"], c["smoothing"]
    on = st["ids"] >= 0
    at = st["ids"].long().clamp(min=0)
    Wf, hf = st["W"].float(), st["h"].float()
    z = hf @ Wf.t()
    m = z.amax(dim=1)
    e = torch.exp(z - m[:, None])
    total = e.sum(dim=1)
    lse = m + torch.log(total)
    mean_z = z.sum(dim=1) / V if eps > 0 else None
    nll = -_of_target(z, at)
    loss = (1 - eps) * nll
    if eps > 0:
        loss = loss + eps * (lse - mean_z)
    zero = torch.zeros_like(loss)
    losses = torch.where(on, loss + c["z_loss"] * lse * lse, zero)
    count = on.sum().clamp(min=1)

    def mean(x):
        return torch.where(on, x, zero).sum(dtype=torch.float64) / count

    share = 1.0 / count.double() if c["reduction"] == "mean" else torch.ones_like(count, dtype=torch.float64)
    stats = torch.stack([losses.sum(dtype=torch.float64) * share, mean(nll), mean(lse * lse)]).float()
    out = dict(stats=stats, losses=losses)
    if not c["grads"]:
        return out
    up = torch.where(on, share.float().expand_as(loss), zero)
    lift = 1.0 + 2.0 * c["z_loss"] * lse  # d(lse + z_loss lse^2) / d lse
    dz = e * (lift / total * up)[:, None] - (eps / V * up)[:, None]
    # p_y - 1 from the log-probability: it cancels where the target is likely
    own_term = torch.expm1(-nll) + (lift - 1.0) * torch.exp(-nll) + eps * (1.0 - 1.0 / V)
    dz.scatter_(1, at[:, None], (own_term * up)[:, None])
    return dict(out, grad_h=(dz @ Wf).to(torch.bfloat16), grad_W=(dz.t() @ hf).to(torch.bfloat16))


def work(case):
    op, V, D = case["op"], case["V"], case["D"]
    scales = math.ceil(V / BLOCK) * math.ceil(D / BLOCK)
    if op == "quantize":
        return {"bytes": 3 * V * D + scales, "flops": 2 * V * D}
    B = case["B"]
    if op == "xent":
        rows = round(B * (1.0 - case["ignore"]))
        if not case["grads"]:
            return {"bytes": 2 * V * D + 2 * rows * D + 8 * B, "flops": 2 * rows * V * D}
        return {"bytes": 4 * V * D + 2 * rows * D + 2 * B * D + 8 * B, "flops": 6 * rows * V * D}
    out = {"logits": B * V * (4 if case.get("dtype") == "fp32" else 2), "sample": 12 * B,
           "logprob": 16 * B}[op]
    return {"bytes": V * D + scales + 2 * B * D + out, "flops": 2 * B * V * D}


# ---------------------------------------------------------------------------
# the definitions in fp64
# ---------------------------------------------------------------------------
def _exact_e4m3(x, rows):
    """(values, scales) of x's blocks in fp64."""
    R, D = x.shape
    v = torch.zeros(-(-R // rows) * rows, -(-D // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    v[:R, :D] = x
    v = v.reshape(-1, rows, v.shape[1] // BLOCK, BLOCK)
    top = v.abs().amax(dim=3).amax(dim=1)
    e = torch.ceil(torch.log2(top / 448.0))
    # log2 is near an integer at the border: settle it by the values themselves
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(top > 0, e.clamp(min=-110.0), torch.zeros_like(e))
    scale = torch.exp2(e)
    y = v / scale[:, None, :, None]
    binade = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    y = torch.round(y / binade) * binade
    return y.reshape(-1, y.shape[2] * BLOCK)[:R, :D], scale


def _exact_values(x, rows):
    y, scale = _exact_e4m3(x, rows)
    R, D = y.shape
    return y * scale.repeat_interleave(rows, 0)[:R].repeat_interleave(BLOCK, 1)[:, :D]


def exact(case, seed):
    global own
    was, own = own, False  # the inputs alone: nothing laid out by the library
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op, V, D = case["op"], case["V"], case["D"]
    if op == "quantize":
        y, scale = _exact_e4m3(st["W"], BLOCK)
        if case["packed"]:
            full = torch.zeros(-(-V // 16) * 16, D, dtype=torch.float64, device=y.device)
            full[:V] = y
            y = full.reshape(-1, 16, D // 64, 4, 16).permute(0, 2, 3, 1, 4).flatten()
        return dict(q=y, scale=scale)
    if op == "xent":
        return _exact_xent(case, st)
    z = torch.matmul(_exact_values(st["h"], 1), _exact_values(st["W"], BLOCK).transpose(0, 1))
    if op == "logits":
        return dict(logits=z)
    beta = torch.tensor([float(torch.tensor(1.0) / torch.tensor(t)) if t > 0 else 1.0
                         for t in st["T"].tolist()], dtype=torch.float64, device=z.device)
    if op == "sample":
        g = _noise(case["B"], V, case["offset"], st["seed"], st["step"], z.device)
        s = torch.where((st["T"] > 0)[:, None], z * beta[:, None] + g, z)
        return dict(ids=s.argmax(dim=1).to(torch.int32) + case["offset"], maxval=s.amax(dim=1))
    z *= beta[:, None]
    lse = torch.logsumexp(z, dim=1)
    lp = []
    for b, t in enumerate(st["ids"].tolist()):
        t -= case["offset"]
        if st["ids"][b] < 0:
            lp.append(torch.zeros_like(lse[0]))
        elif 0 <= t < V:
            others = torch.logsumexp(torch.cat([z[b, :t], z[b, t + 1:]]), dim=0)
            lp.append(-torch.logaddexp(others - z[b, t], torch.zeros_like(lse[0])))
        else:
            lp.append(torch.full_like(lse[0], -math.inf))
    return dict(logprob=torch.stack(lp), lse=lse)


def _exact_xent(case, st):
    """Row by row blocks; a row's log-probability as log(p_y) with p_y = 1 - the
    others' share."""
    V, B, s, lam = case["V"], case["B"], case["smoothing"], case["z_loss"]
    h, W = st["h"].double(), st["W"].double()
    ids = st["ids"].long()
    keep = (ids >= 0).nonzero()[:, 0]
    n = max(1, len(keep))
    share = 1.0 / n if case["reduction"] == "mean" else 1.0
    losses = torch.zeros(B, dtype=torch.float64, device=h.device)
    gh, gw = torch.zeros_like(h), torch.zeros_like(W) if case["grads"] else None
    nll_sum = sq_sum = 0.0
    step = max(1, (1 << 27) // V)
    for r in range(0, len(keep), step):
        rows = keep[r:r + step]
        y = ids[rows]
        z = torch.matmul(h[rows], W.transpose(0, 1))
        lse = torch.logsumexp(z, dim=1)
        p = torch.softmax(z, dim=1)
        hot = torch.zeros_like(z).scatter_(1, y.unsqueeze(1), 1.0)
        others = (p * (1.0 - hot)).sum(dim=1)
        nll = torch.where(others < 0.5, -torch.log1p(-others), lse - (z * hot).sum(dim=1))
        losses[rows] = (1 - s) * nll + s * (lse - z.mean(dim=1)) + lam * lse ** 2
        nll_sum += float(nll.sum())
        sq_sum += float((lse ** 2).sum())
        if case["grads"]:
            lift = (1.0 + 2.0 * lam * lse).unsqueeze(1)
            dz = lift * p - s / V
            mine = -others + (lift[:, 0] - 1.0) * (1.0 - others) + s - s / V
            dz = torch.where(hot > 0, mine.unsqueeze(1), dz) * share
            gh[rows] = torch.matmul(dz, W)
            gw += torch.matmul(dz.transpose(0, 1), h[rows])
    stats = torch.tensor([float(losses.sum()) * share, nll_sum / n, sq_sum / n], dtype=torch.float64)
    out = dict(stats=stats, losses=losses)
    return dict(out, grad_h=gh, grad_W=gw) if case["grads"] else out
