"""The codes of the device error record (no GPU): the calls that may run at once in a training or serving
process share one record, so a code of the packed kernels names one wait of one kernel."""
import os
import re
from collections import Counter

from exact_io_aware_16_gb300 import build as fabuild


def codes(name):
    """The codes of the waits of a file: literals with a role's digit and two more, behind a kernel's digit or none."""
    with open(os.path.join(fabuild.CSRC, name)) as f:
        return Counter(int(x, 16) for x in re.findall(r"\b0x([1-9]?[1-57][0-9a-f]{2})\b(?=[),;])", f.read()))


def test_a_code_of_the_packed_kernels_names_one_wait():
    others = set().union(*(codes(s) for s in fabuild.SOURCES if not s.startswith("fa_packed")), {0x7e0})
    assert len(others) > 50
    packed, backward = codes("fa_packed.cu"), codes("fa_packed_bwd.cu")
    assert len(packed) > 12 and len(backward) > 30
    assert max((packed + backward).values()) == 1
    assert not others & set(packed) and not others & set(backward)
    # the kernel's digit: 1 the forward pass, 2 dq, 3 dk and dv
    assert {c >> 12 for c in packed} == {1} and {c >> 12 for c in backward} == {2, 3}
