"""Code-generation check of the products' stores (host only: compiles the translation unit
to gfx950 assembly and reads it): the kernels of dW that pass the caches do so with every
store of a row's stretch, the others with none."""
import re

import pytest

import test_codegen_tiles as tiles

pytestmark = tiles.pytestmark


def test_stores_of_dW_pass_the_caches_or_not(tmp_path):
    s = tiles._assemble("fs_logprob_grad.hip", str(tmp_path))
    seen = []
    for n in re.findall(r"^\s*\.amdhsa_kernel (\S+)", s, re.M):
        if "grad_weights_kernel" not in n:
            continue
        start = s.index("\n" + n + ":")
        body = s[start:s.index(".Lfunc_end", start)]
        stores = re.findall(r"global_store_dwordx4 .*", body)
        hinted = sum(bool(re.search(r"\bnt\b", x)) for x in stores)
        wa, wb, mr, nt = (int(x) for x in re.search(r"4TileILi\d+ELi\d+ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)", n).groups())
        whole = nt * 16 * mr * 16 // (8 * 64)      # 16 bytes per lane of a wave's part of dW
        seen.append(hinted)
        assert hinted in (0, whole), f"{n}: {hinted} of {whole} stores"
    assert any(seen) and not all(seen), seen
