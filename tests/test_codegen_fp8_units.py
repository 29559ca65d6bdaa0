"""Code-generation checks of the 8-bit head's streaming logits and quantising kernels
(host only: compiles their translation units to gfx950 assembly and reads it): registers
hold everything."""
import pytest

import test_codegen_head as head

pytestmark = head.pytestmark


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    units, head.UNITS = head.UNITS, ("fs_fp8_stream_logits.hip", "fs_fp8_quantize.hip")
    try:
        return head.kernels.__wrapped__(tmp_path_factory)
    finally:
        head.UNITS = units


def test_registers_hold_everything(kernels):
    assert len([n for n in kernels if "fp8_stream_kernel" in n]) == 40   # both types of logits
    assert len([n for n in kernels if "quantize" in n or "pack_fp8" in n]) == 5
    for name, (_, scratch) in kernels.items():
        assert scratch == 0, f"{name}: {scratch} bytes of scratch"
