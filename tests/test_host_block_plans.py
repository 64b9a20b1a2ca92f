"""Work plans of listed blocks and shared prefixes (host arithmetic, no GPU): what they cost."""
import os
import subprocess
import sys

import pytest

from paged_mla_kv_gb300 import build as BUILD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()


# The largest batches that the calls take: a plan holds runs of equal units, so it takes neither their memory
# nor their time.
@pytest.mark.parametrize("call", [
    "B.tf_paged_mla_blocks_workspace_bytes(None, 1, 1 << 30, 1, [1 << 30], 1)",
    "B.tf_paged_mla_blocks_workspace_bytes(None, 1, 1 << 30, 1, [(1 << 31) - 1], 4096)",
    "B.tf_paged_mla_blocks_workspace_bytes(None, 512, 1 << 14, 128, [1 << 20] * 512, 100)",
    "B.tf_paged_mla_shared_workspace_bytes(None, 2, 1 << 22, 128, [1 << 30] * 2, [2], [1 << 20])"])
def test_the_largest_plans_are_small(call):
    code = ("import resource, time\nfrom paged_mla_kv_gb300 import binding as B\n"
            "B.tf_paged_mla_blocks_workspace_bytes(None, 1, 1, 16, [64], 8)\n"
            "a, t = resource.getrusage(resource.RUSAGE_SELF).ru_maxrss, time.perf_counter()\n"
            f"n = {call}\n"
            "t = time.perf_counter() - t\nprint(n, resource.getrusage(resource.RUSAGE_SELF).ru_maxrss - a, t)")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-500:]
    n, kib, seconds = r.stdout.split()
    assert int(n) >= 0 and int(kib) < 8192 and float(seconds) < 0.25, r.stdout
