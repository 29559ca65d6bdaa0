"""Plain reference of the 8-bit LM head (test infrastructure), on the CPU and from
the format's definition; shares no code with the library.

A quantised value times its power of two has four significant bits, so the
dequantised tensors are exact in bf16: every reference of the bf16 head (logits,
log-probabilities, the sampler's oracle) is one of the 8-bit head on them."""
import math

import torch

F64 = torch.float64
BLOCK = 128


def e4m3_table():
    """The finite magnitudes of e4m3, by code 0 .. 126."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append((1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6)
    return torch.tensor(out, dtype=F64)


def round_e4m3(x):
    """Codes of the nearest e4m3 values (ties to the even code) of finite |x| <= 448."""
    t = e4m3_table()
    a = x.abs().to(F64)
    hi = torch.searchsorted(t, a).clamp(max=126)       # first value >= a
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - t[lo], t[hi] - a
    take_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    code = torch.where(take_hi, hi, lo)
    return code + torch.where(torch.signbit(x), 128, 0)


def quantise(x, rows):
    """(codes uint8, scale bytes uint8) of a bf16 matrix in blocks of rows x 128."""
    R, D = x.shape
    VB, KB = -(-R // rows), -(-D // BLOCK)
    codes = torch.zeros(R, D, dtype=torch.int64)
    scales = torch.zeros(VB, KB, dtype=torch.int64)
    x = x.to(F64)
    for i in range(VB):
        for k in range(KB):
            b = x[i * rows:(i + 1) * rows, k * BLOCK:(k + 1) * BLOCK]
            fin = torch.isfinite(b)
            top = float(torch.where(fin, b.abs(), torch.zeros_like(b)).max())
            e = 0
            if top > 0:
                e = -110
                while top > math.ldexp(448.0, e):
                    e += 1
            scales[i, k] = e + 127
            c = round_e4m3(torch.where(fin, b, torch.zeros_like(b)) * 2.0 ** -e)
            codes[i * rows:(i + 1) * rows, k * BLOCK:(k + 1) * BLOCK] = torch.where(fin, c, 0x7F)
    return codes.to(torch.uint8), scales.to(torch.uint8)


def dequantise(codes, scales, rows):
    """bf16 values (exact for scales of 2^-110 and more)."""
    t = torch.cat([e4m3_table(), torch.tensor([math.nan], dtype=F64)])
    c = codes.long()
    v = t[c & 127] * torch.where(c >= 128, -1.0, 1.0).to(F64)
    s = torch.pow(2.0, scales.to(F64) - 127)
    R, D = codes.shape
    v = v * s.repeat_interleave(rows, 0)[:R].repeat_interleave(BLOCK, 1)[:, :D]
    return v.to(torch.bfloat16)


def pack(codes):
    """Row-major codes in fragment order, byte by byte from its definition."""
    V, D = codes.shape
    G, S = -(-V // 16), D // 64
    out = torch.zeros(G * S * 64 * 16, dtype=torch.uint8)
    i = torch.arange(out.numel())
    j, l, gs = i % 16, i // 16 % 64, i // 1024
    s, g = gs % S, gs // S
    v, k = 16 * g + l % 16, 64 * s + 16 * (l // 16) + j
    inside = v < V
    out[inside] = codes[v[inside], k[inside]]
    return out


def matrix_rounding(h, W):
    """What the 8-bit matrix instructions add to a logit's error, on values without
    a pattern.  They align the products of eight neighbouring k to the largest
    exponent sum E among them and cut each below 2^(E - 12): an error uniform in (0,
    2^(E - 12)) with the product's sign, of variance 2^(2 E - 24) / 3.  E is at
    most the sum of the eight's largest exponents (2^-6 in a block's units for
    subnormal values).  Six deviations of the sum over a row."""
    def tops(codes, scales, rows):
        R, D = codes.shape
        t = torch.cat([e4m3_table(), torch.zeros(1, dtype=F64)])
        v = t[codes.long() & 127].clamp(min=2.0 ** -6)
        v = torch.pow(2.0, torch.floor(torch.log2(v)))
        s = torch.pow(2.0, scales.to(F64) - 127)
        v = v * s.repeat_interleave(rows, 0)[:R].repeat_interleave(BLOCK, 1)[:, :D]
        return v.reshape(R, D // 8, 8).amax(dim=2)
    a, b = tops(*h, 1), tops(*W, BLOCK)
    return 6 * math.sqrt(8 / 3) * 2.0 ** -12 * ((a ** 2) @ (b ** 2).T).sqrt()
