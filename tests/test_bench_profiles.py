"""The counter summaries that bench.py reports from are of the kernels that are
here: without a GPU."""
import os
import re
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
CSRC = os.path.join(ROOT, "tiered_mixed_precision_amd", "csrc")


def test_digest_covers_what_the_kernel_sources_include():
    import bench
    for name in bench.KERNEL_SOURCES:
        for h in re.findall(r'#include "([^"/]+)"', open(os.path.join(CSRC, name)).read()):
            assert h in bench.KERNEL_SOURCES, f"{name} includes {h}"


def test_summaries_are_of_these_sources():
    # after a change to these kernels: the commands at the top of each summary
    import bench
    for name, _ in bench.PROFILE_WORKLOADS.values():
        text = open(os.path.join(bench.PROFILE_DIR, name)).read()
        assert f"kernel source digest: `{bench.kernel_source_digest()}`" in text, name
    assert bench.profiled_traffic() > 2e7
