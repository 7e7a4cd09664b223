"""What reading the device error record copies: nothing for packed kernels that never ran in the process."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import torch
from torch.profiler import ProfilerActivity, profile
import exact_io_aware_16_gb300 as fa

x = torch.zeros(8, 1, 64, dtype=torch.bfloat16, device="cuda")
cu = torch.tensor([0, 8], dtype=torch.int32, device="cuda")

def copies():
    with profile(activities=[ProfilerActivity.CPU, ProfilerActivity.CUDA]) as p:
        assert fa.fa_get_device_error() == (0, 0)
        torch.cuda.synchronize()
    return sum("Memcpy DtoH" in e.name for e in p.events())

fa.fa_get_device_error()
copies()
before = copies()
o, lse = fa.fa_forward_packed(x, x, x, cu)
forward = copies()
fa.fa_backward_packed(x, x, x, o, x, lse, cu)
print(before, forward, copies())
"""


def test_records_of_packed_kernels_are_copied_once_they_have_run():
    from exact_io_aware_16_gb300 import build

    build.build()
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    before, forward, both = map(int, r.stdout.split()[-3:])
    if before == 0:
        pytest.skip("the profiler records no copies here")
    assert forward == before + 1 and both == before + 2
