"""Code-generation checks of the block-tiled training kernels (host only:
compiles their translation units to gfx950 assembly and reads it).

The main loop stages both operands into LDS with direct global->LDS loads and
waits for them by counting vector-memory operations in issue order, so no other
vector-memory operation may be issued between the first staging load and the
last wait, and every barrier must follow a wait that covers the tile it
publishes and the LDS reads of the slot it frees.  Fragments and accumulators
must stay in registers."""
import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "lm_head_exact_amd", "csrc")
UNITS = ("fs_logprob.hip", "fs_logprob_grad.hip")

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None and
                                not os.path.exists("/opt/rocm/bin/hipcc"), reason="needs hipcc")


def _assemble(unit, outdir):
    from lm_head_exact_amd import build
    out = os.path.join(outdir, unit + ".s")
    r = subprocess.run([build.HIPCC, *build.FLAGS, "-S", "--cuda-device-only",
                        os.path.join(CSRC, unit), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return open(out).read()


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Assembly lines of every kernel over a Tile, by demangled name, and its scratch bytes."""
    outdir = str(tmp_path_factory.mktemp("asm"))
    with ThreadPoolExecutor(2) as ex:
        texts = list(ex.map(lambda u: _assemble(u, outdir), UNITS))
    found = {}
    for s in texts:
        names = re.findall(r"^(_Z\S*4Tile\S*):", s, re.M)
        plain = subprocess.run(["c++filt"], input="\n".join(names), capture_output=True,
                               text=True).stdout.splitlines()
        for n, d in zip(names, plain):
            start = s.index("\n" + n + ":")
            body = s[start:s.index(".Lfunc_end", start)].splitlines()
            meta = s[s.index(".amdhsa_kernel " + n):]
            scratch = int(re.search(r"private_segment_fixed_size (\d+)", meta).group(1))
            found[d] = (body, scratch)
    assert len(found) >= 20, sorted(found)
    return found


def _shape(name):
    m = re.search(r"Tile<(\d+), (\d+), (\d+), (\d+), (\d+), (\d+), (\d+), (\d+)", name)
    assert m, name
    _, _, wa, wb, mr, nt, s, bk = (int(x) for x in m.groups())
    ta, tb, nw = wa * mr * 16, wb * nt * 16, wa * wb
    return s, (ta + tb) * bk * 2 // (nw * 1024)   # ring slots, staging loads per wave and tile


def _events(lines):
    """L staging load, G other vector-memory operation, (vm, lgkm) wait, B barrier."""
    for line in lines:
        t = line.strip()
        if re.match(r"buffer_load\S* .*\blds\b", t):
            yield "L"
        elif re.match(r"(buffer|global|flat|scratch)_(load|store|atomic)", t):
            yield "G"
        elif t.startswith("s_waitcnt"):
            vm, lgkm = re.search(r"vmcnt\((\d+)\)", t), re.search(r"lgkmcnt\((\d+)\)", t)
            yield (int(vm.group(1)) if vm else None, int(lgkm.group(1)) if lgkm else None)
        elif t.startswith("s_barrier"):
            yield "B"


def test_waits_cover_what_the_barriers_publish(kernels):
    for name, (lines, _) in kernels.items():
        slots, loads = _shape(name)
        ev = list(_events(lines))
        first = ev.index("B")
        before = ev[:first]
        start = before.index("L")
        assert all(e != "G" for e in before[start:]), f"{name}: another load among the first tiles'"
        assert before.count("L") == slots * loads, f"{name}: {before.count('L')} prologue loads"
        waits = [e for e in before[start:] if isinstance(e, tuple) and e[0] is not None]
        assert waits and waits[-1][0] <= (slots - 1) * loads, f"{name}: prologue wait {waits}"
        # the main loop: up to the next vector-memory operation that is no staging load
        rest = ev[first + 1:]
        end = rest.index("G") if "G" in rest else len(rest)
        loop, since, barriers = rest[:end], [], 0
        for e in loop:
            if e == "B":
                vm = [w[0] for w in since if isinstance(w, tuple) and w[0] is not None]
                lg = [w[1] for w in since if isinstance(w, tuple) and w[1] is not None]
                assert vm and vm[-1] <= (slots - 2) * loads, f"{name}: barrier after {since}"
                assert lg and lg[-1] == 0, f"{name}: barrier with LDS reads in flight {since}"
                since, barriers = [], barriers + 1
                last = vm[-1]
            else:
                since.append(e)
        assert barriers >= 2 and last == 0, f"{name}: {barriers} barriers, last wait {last}"
        staged = [e for e in loop if e == "L"]
        assert len(staged) % loads == 0 and staged, f"{name}: {len(staged)} loop loads"


def test_transposing_reads_do_not_wait_for_the_loads_in_flight(kernels):
    """The slot read and the slot refilled are distinct; a wait for all loads
    before each read would serialise them."""
    seen = 0
    for name, (lines, _) in kernels.items():
        slots, loads = _shape(name)
        if slots < 3 or not any("ds_read_b64_tr_b16" in x for x in lines):
            continue
        first = next(i for i, x in enumerate(lines) if x.strip().startswith("s_barrier"))
        body = lines[first:]
        loop = [x.strip() for x in body[:next((i for i, x in enumerate(body) if re.match(
            r"\s*(global|flat)_(load|store)", x)), len(body))]]
        zero = [x for x in loop if x.startswith("s_waitcnt") and "vmcnt(0)" in x]
        assert len(zero) <= 1, f"{name}: {len(zero)} waits for every load"
        seen += 1
    assert seen >= 3


def test_registers_hold_everything(kernels):
    for name, (_, scratch) in kernels.items():
        assert scratch == 0, f"{name}: {scratch} bytes of scratch"
