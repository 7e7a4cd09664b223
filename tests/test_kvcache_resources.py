"""Register and spill budget of the key/value cache's kernels, from the compiler's own
report of the sources as built (no GPU).

The tree decode runs two CTAs an SM up to 32 query rows a key head and one with 64; its
registers a thread have to leave room for them.  The tile loop of 16 rows spills nothing.
With 32 and 64 rows a thread is at the limit that 10 and 19 or 18 warps leave it, and what
the loop does not need lies in a few dozen bytes of local memory: bounded here, so that
a change that spills the loop itself shows.  The writer, reader, commit and merge spill
nothing.
"""
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from exact_io_aware_16_gb300 import build as fabuild
from test_kernel_resources import parse

SOURCES = ("fa_tree.cu", "fa_cache.cu")
TREE = re.compile(r"fa_tree_kernelILi(\d+)ELb([01])ELi(\d+)E")
OTHERS = ("fa_tree_combine", "fa_cache_write_kernel", "fa_cache_read_kernel", "fa_cache_commit_kernel")


@pytest.fixture(scope="module")
def report(tmp_path_factory):
    try:
        cc = fabuild.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not found")
    out = tmp_path_factory.mktemp("ptxas")

    def one(src):
        cmd = [cc, *fabuild.ARCH, *fabuild.FLAGS, "-Xptxas", "-v", "-c", os.path.join(fabuild.CSRC, src),
               "-o", str(out / (src + ".o"))]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        return r.stdout + r.stderr

    with ThreadPoolExecutor(len(SOURCES)) as ex:
        entries = parse("\n".join(ex.map(one, SOURCES)))
    return {n: st for n, st in entries.items() if "regs" in st}


def test_tree_kernels(report):
    seen = {}
    for name, st in report.items():
        m = TREE.search(name)
        if m:
            seen[int(m[1]), m[2] == "1", int(m[3])] = st
    assert set(seen) == {(d, f8, nr) for d in (64, 128) for f8 in (False, True) for nr in (16, 32, 64)}
    for (d, f8, nr), st in seen.items():
        tag = f"<{d}, {'e4m3' if f8 else 'bf16'}, {nr}>: {st}"
        ctas = 1 if nr == 64 else 2
        threads = 8 * nr + 32 + 32 * (2 if ctas == 1 else 1)
        assert st["regs"] * threads * ctas <= 65536, tag
        if nr == 16:
            assert st["spill_st"] == 0 and st["spill_ld"] == 0, tag
        else:
            assert st["spill_st"] <= 96 and st["spill_ld"] <= 48, tag


def test_the_other_kernels_spill_nothing(report):
    for kernel in OTHERS:
        found = [st for n, st in report.items() if kernel in n]
        assert len(found) == 4, kernel
        for st in found:
            assert st["spill_st"] == 0 and st["spill_ld"] == 0 and st["stack"] == 0, (kernel, st)
