"""A workspace size is host arithmetic: it makes no context on the GPU, and what it found does not decide later calls."""
import subprocess
import sys

import pytest

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD

pytestmark = pytest.mark.gpu

CODE = """
import ctypes
from paged_mla_kv_gb300 import binding as B

cu = ctypes.CDLL("libcuda.so.1")
assert cu.cuInit(0) == 0

def active():
    flags, on = ctypes.c_uint(0), ctypes.c_int(0)
    assert cu.cuDevicePrimaryCtxGetState(0, ctypes.byref(flags), ctypes.byref(on)) == 0
    return on.value

lens = [32768] * 64
assert active() == 0
assert B.tf_paged_mla_workspace_bytes(None, 64, 1, 64, lens) > 0
assert active() == 0
assert B.tf_paged_mla_blocks_workspace_bytes(None, 64, 1, 64, lens, 32) > 0
assert B.tf_paged_mla_blocks_workspace_bytes(None, 1, 1, 16, [2048], 8) > 0
assert B.tf_paged_mla_shared_workspace_bytes(None, 64, 1, 64, lens, [64], [512]) > 0
assert active() == 0
print("sized")
"""


def test_workspace_sizes_make_no_context():
    BUILD.build()
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "sized", r.stderr[-2000:]
