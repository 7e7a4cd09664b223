"""Register and spill budget of the packed attention's and the rotation's kernels, from the
compiler's own report of the sources as built (no GPU).

One CTA of the attention kernels fills an SM: eight warps of softmax or gradient, one of copies
and two or three that issue products; registers are allotted to warps in fours.  None of them
spills.  The norm's kernels hold a row, its weights and the next row's
load, and may leave up to four registers of addresses in local memory.
"""
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from exact_io_aware_16_gb300 import build as fabuild
from test_kernel_resources import parse

SOURCES = ("fa_packed.cu", "fa_packed_bwd.cu", "fa_rotary.cu")


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


def found(report, pattern):
    return {tuple(int(x) for x in m.groups()): st
            for n, st in report.items() for m in [re.search(pattern, n)] if m}


def allotted(regs, warps):
    """Registers of a CTA: by the warp in units of 256, warps in fours."""
    return -(-regs * 32 // 256) * 256 * (-(-warps // 4) * 4)


def test_packed_forward(report):
    seen = found(report, r"fa_packed_fwd_kernelILi(\d+)ELb([01])E")
    assert set(seen) == {(d, c) for d in (64, 128) for c in (0, 1)}
    for key, st in seen.items():
        assert allotted(st["regs"], 11) <= 65536, (key, st)
        assert st["spill_st"] == 0 and st["spill_ld"] == 0 and st["stack"] == 0, (key, st)


def test_packed_backward_and_plan_spill_nothing(report):
    shapes = {(64, c, 1) for c in (0, 1)} | {(128, c, n) for c in (0, 1) for n in (1, 2)}
    for kernel in ("fa_packed_dq_kernel", "fa_packed_dkdv_kernel"):
        seen = found(report, kernel + r"ILi(\d+)ELb([01])ELi(\d+)E")
        assert set(seen) == shapes, kernel
        for key, st in seen.items():
            assert allotted(st["regs"], 12) <= 65536, (kernel, key, st)
            assert st["spill_st"] == 0 and st["spill_ld"] == 0 and st["stack"] == 0, (kernel, key, st)
    (plan,) = found(report, r"(?:)fa_packed_plan_kernel").values()
    assert plan["spill_st"] == 0 and plan["spill_ld"] == 0 and plan["stack"] == 0, plan


def test_rotary_and_norm(report):
    seen = found(report, r"fa_rotary_kernelILi(\d+)ELi(\d)E")
    assert set(seen) == {(d, mode) for d in (64, 128) for mode in range(4)}
    for (d, mode), st in seen.items():
        most = 0 if mode < 2 else 32  # modes 2 and 3 are the norm's
        assert st["spill_st"] <= most and st["spill_ld"] <= most, (d, mode, st)
    for d, st in found(report, r"fa_norm_weight_kernelILi(\d+)E").items():
        assert st["spill_st"] == 0 and st["spill_ld"] == 0, (d, st)
