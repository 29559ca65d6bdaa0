"""The reference of the 8-bit head against independent facts (CPU)."""
import math

import pytest
import torch

import fp8_ref

F64 = torch.float64


def test_rounding_against_torch():
    """Every bf16 value that is finite and at most 448: the nearest e4m3, ties to even."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16)
    x = x[torch.isfinite(x) & (x.abs() <= 448)]
    assert torch.equal(fp8_ref.round_e4m3(x.to(F64)).to(torch.uint8), x.to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("R,D,rows", [(1, 64, 1), (5, 320, 1), (130, 192, 128), (300, 128, 128)])
def test_scales_are_the_least(R, D, rows):
    g = torch.Generator().manual_seed(R + D)
    x = (torch.randn(R, D, generator=g) * torch.exp(4 * torch.randn(R, 1, generator=g))).to(torch.bfloat16)
    codes, scales = fp8_ref.quantise(x, rows)
    v = fp8_ref.dequantise(codes, scales, rows).to(F64)
    assert torch.isfinite(v).all()
    for i in range(scales.shape[0]):
        for k in range(scales.shape[1]):
            b = x[i * rows:(i + 1) * rows, k * 128:(k + 1) * 128].to(F64)
            s = 2.0 ** (int(scales[i, k]) - 127)
            assert 224 * s < float(b.abs().max()) <= 448 * s
            err = (v[i * rows:(i + 1) * rows, k * 128:(k + 1) * 128] - b).abs()
            # half a step: 2^-4 of the value, or 2^-10 scales among the smallest
            assert (err <= torch.clamp(b.abs() * 2.0 ** -4, min=s * 2.0 ** -10)).all()


def test_special_blocks():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    x[1, 3] = math.inf
    x[1, 4] = 2.0
    x[2, 5] = math.nan
    x[3, 0] = 2.0 ** -133
    codes, scales = fp8_ref.quantise(x, 1)
    assert scales[:, 0].tolist() == [127, 127 - 7, 127, 127 - 110]
    assert codes[1, 3] == 0x7F and codes[2, 5] == 0x7F and int(codes[0].max()) == 0


def test_fragment_order_of_one_group():
    codes = torch.arange(16 * 128).remainder(251).to(torch.uint8).view(16, 128)
    p = fp8_ref.pack(codes).view(2, 4, 16, 16)   # step, quarter of 64 columns, row, byte
    for s in range(2):
        for c in range(4):
            assert torch.equal(p[s, c], codes[:, 64 * s + 16 * c:64 * s + 16 * c + 16])
