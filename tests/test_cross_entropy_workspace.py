"""fs_cross_entropy's workspace with gradients serves the loss alone of the same sizes
(host only): a training loop that allocates once evaluates with the same buffer."""
import pytest

import lm_head_exact_amd as fs
from lm_head_exact_amd import binding

SIZES = [1, 2, 8, 15, 16, 17, 31, 32, 33, 64, 65, 100, 127, 128, 129, 256, 513, 2000]


@pytest.mark.parametrize("D", [8, 64, 72, 256, 264, 1024, 4096, 5120, 5128, 8192, 8200, 16384])
def test_gradients_take_no_less(D):
    L = binding.lib()
    for B in SIZES:
        for V in SIZES + [300, 1000, 8192, 8193, 16032, 32000, 32768, 32769, 128256]:
            grads = L.fs_cross_entropy_workspace_bytes(B, D, V, 1)
            alone = L.fs_cross_entropy_workspace_bytes(B, D, V, 0)
            assert 0 < alone <= grads, (B, D, V, alone, grads)


@pytest.mark.parametrize("V", [1, 16, 17, 300])
def test_few_entries_take_few_partials(V):
    """One pair per row and 16 vocabulary rows at most (and one of a group that starts in
    the middle) and what is rounded up to 256 bytes, twice."""
    for B, D in ((1, 64), (16, 8192), (32, 5120)):
        groups = (V + 3 + 15) // 16
        assert fs.token_logprobs_workspace_bytes(B, D, V) <= 8 * groups * B + 4 * B + 512
        assert fs.fp8_workspace_bytes(B, D, V) <= 8 * groups * B + 4 * B + 512
