"""The binding on a torch without the scales' 8-bit type (host only): what does not need
it is there, and what does says so."""
import importlib.util
import sys

import pytest
import torch

from lm_head_exact_amd import binding


@pytest.fixture
def without_e8m0(monkeypatch):
    monkeypatch.delattr(torch, "float8_e8m0fnu")
    name = "lm_head_exact_amd._binding_without_e8m0"
    spec = importlib.util.spec_from_file_location(name, binding.__file__)
    module = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(sys.modules, name, module)
    spec.loader.exec_module(module)
    return module


def test_bf16_calls_do_not_need_the_scales_type(without_e8m0):
    b = without_e8m0
    h, W = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(10, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="(?i)device|gpu|cuda"):   # (as with it: host tensors are refused)
        b.cross_entropy(h, W, torch.zeros(2, dtype=torch.int32))
    assert b.token_logprobs_workspace_bytes(4, 64, 100) > 0
    assert b.fp8_workspace_bytes(4, 64, 100) > 0


def test_calls_that_need_it_say_so(without_e8m0, monkeypatch):
    b = without_e8m0
    monkeypatch.setattr(b, "_req", lambda *a, **k: None)   # (no device here)
    h, W = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(10, 64, dtype=torch.bfloat16)
    q = torch.zeros(16 * 64, dtype=torch.float8_e4m3fn)
    s = torch.zeros(1, 1, dtype=torch.uint8)
    with pytest.raises(RuntimeError, match="float8_e8m0fnu"):
        b.quantize_weights_fp8(W)
    with pytest.raises(RuntimeError, match="float8_e8m0fnu"):
        b.logits_fp8(h, q, s, 10)
    with pytest.raises(RuntimeError, match="float8_e8m0fnu"):
        b.token_logprobs_fp8(h, q, s, 10, None, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(RuntimeError, match="float8_e8m0fnu"):
        b.sample_fp8(h, q, s, 10, torch.ones(2), 1, 2)
