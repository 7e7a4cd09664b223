"""What keeps the library's kernels legal in runs of several GPUs (no GPU needed)."""
import glob
import os

from exact_io_aware_16_gb300 import build as fabuild


def test_no_source_loads_or_commits_by_multicast():
    """TMA copies and commits reach the block that issues them alone."""
    files = glob.glob(os.path.join(fabuild.CSRC, "*.cu*")) + glob.glob(os.path.join(fabuild.CSRC, "*.h"))
    assert len(files) >= len(fabuild.SOURCES) + len(fabuild.HEADERS)
    for f in files:
        with open(f) as src:
            assert "multicast" not in src.read(), os.path.basename(f)
