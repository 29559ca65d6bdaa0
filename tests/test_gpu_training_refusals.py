"""Calls of the training operators that the binding refuses, or must not (GPU:
the binding checks device tensors; a refused call launches nothing)."""
import ctypes

import pytest
import torch

import lm_head_exact_amd as fs
from lm_head_exact_amd import binding as bd

pytestmark = pytest.mark.gpu


def clip_workspace(grads):
    sizes = (ctypes.c_int64 * len(grads))(*[g.numel() for g in grads])
    return int(bd.lib().fs_clip_grad_norm_workspace_bytes(sizes, len(grads)))


def test_clipping_keeps_norm_and_workspace_apart_from_the_tensors():
    big = torch.ones(40000).cuda()
    a, b = big[:1000], big[2000:9000]
    grads = [a, b]
    n = clip_workspace(grads)
    for kw in (dict(norm=a[:1]), dict(norm=b[6999:]), dict(workspace=big[2000:9000]),
               dict(workspace=big), dict(out=[torch.empty_like(a), big[20000:27000]], norm=big[26999:27000]),
               dict(out=[big[20000:21000], torch.empty_like(b)], workspace=big[20992:30000]),
               dict(out=[torch.empty_like(a), torch.empty_like(b)], workspace=big[:8000]),
               dict(norm=big[30000:30001], workspace=big[29952:40000])):
        with pytest.raises(ValueError, match="overlap"):
            fs.clip_grad_norm(grads, 1.0, **kw)
    torch.cuda.synchronize()
    assert (big == 1).all()
    # beside them: fine
    ws = big[9024:9024 + n // 4 + 64]
    off = (-ws.data_ptr() % 256) // 4
    norm = fs.clip_grad_norm(grads, 1e9, norm=big[1500:1501], workspace=ws[off:])
    assert norm.data_ptr() == big[1500:].data_ptr() and abs(float(norm) - 8000 ** 0.5) < 1e-4
    assert (a == 1).all() and (b == 1).all()


def test_sizes_and_offsets_beyond_32_bits():
    """They are refused, not cut to 32 bits."""
    h, W = torch.ones(2, 64).to(torch.bfloat16).cuda(), torch.ones(40, 64).to(torch.bfloat16).cuda()
    ids, z = torch.zeros(2, dtype=torch.int32).cuda(), torch.zeros(2).cuda()
    Wp = fs.pack_weights(W)
    for off in (2**31, 2**32, 2**40, -2**32):
        with pytest.raises(ValueError, match="2\\^31"):
            fs.token_logprobs(h, W, None, ids, vocab_offset=off)
        with pytest.raises(ValueError, match="2\\^31"):
            fs.token_logprobs_backward(h, W, None, ids, z, z, z, vocab_offset=off)
    with pytest.raises(ValueError, match="2\\^31"):
        fs.token_logprobs(h, Wp, None, ids, V=2**32 + 40)
    with pytest.raises(fs.FlashSampleError):
        fs.token_logprobs(h, W, None, ids, vocab_offset=2**31 - 40)
    x = torch.empty(2**32 + 5, device="cuda")
    cu = torch.tensor([0, 2, 5], dtype=torch.int32).cuda()
    with pytest.raises(ValueError, match="2\\^31"):
        fs.policy_loss(x, x, z, cu)
    with pytest.raises(ValueError, match="2\\^31"):
        fs.preference_loss(x, cu)
