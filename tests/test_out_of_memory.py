"""Host memory that runs out inside a call: the call returns TF_E_NOMEM (a size: 0), no exception leaves it.

A preloaded library takes the place of operator new and lets it fail on request.  Each case runs in a process
of its own, which an exception would end."""
import os
import shutil
import subprocess
import sys

import pytest

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAIL_NEW = r"""
#include <cstdlib>
#include <new>
static size_t limit = ~(size_t)0;   // requests of this size and more fail
extern "C" void fail_new(size_t n) { limit = n; }
void *operator new(size_t n) {
    void *p = n >= limit ? nullptr : malloc(n ? n : 1);
    if (!p) throw std::bad_alloc();
    return p;
}
void *operator new(size_t n, const std::nothrow_t &) noexcept { return malloc(n ? n : 1); }
void *operator new(size_t n, std::align_val_t a) {
    void *p = n >= limit ? nullptr : aligned_alloc((size_t)a, (n + (size_t)a - 1) / (size_t)a * (size_t)a);
    if (!p) throw std::bad_alloc();
    return p;
}
void operator delete(void *p, std::align_val_t) noexcept { free(p); }
void operator delete(void *p, size_t, std::align_val_t) noexcept { free(p); }
void operator delete(void *p) noexcept { free(p); }
void operator delete(void *p, size_t) noexcept { free(p); }
"""

HOST = """
import ctypes, os
import numpy as np
from paged_mla_kv_gb300 import binding as B
fail = ctypes.CDLL(os.environ["FAIL_NEW"]).fail_new
fail.argtypes = [ctypes.c_size_t]
BASE = 1 << 40
L = B.lib()

def pool(**kw):
    d = B.make_desc(2, 32, **kw)
    h = ctypes.c_void_p()
    assert L.tf_kvpool_create(ctypes.byref(d), BASE, B.tf_kvpool_bytes(d), ctypes.byref(h)) == 0
    return h

def lens(*n):
    a = np.asarray(n, np.int64)
    keep.append(a)
    return a.ctypes.data

keep = []
plain, inv8, f8 = pool(), pool(invariant=True, fp8=True), pool(fp8=True)
n1, n2 = lens(2048), lens(2048, 2048)
ids = np.zeros(3, np.int32)
assert L.tf_kvpool_take(plain, 3, ids.ctypes.data, None) == 0
g, f = np.asarray([2], np.int32), lens(512)
d = B.make_desc(2, 32)
h = ctypes.c_void_p()
info = B.tf_attend_plan()
W = 1 << 40
"""

# calls that take host memory, up to where they would ask the GPU
CALLS = {
    "create": "L.tf_kvpool_create(ctypes.byref(d), BASE, B.tf_kvpool_bytes(d), ctypes.byref(h))",
    "release": "L.tf_kvpool_release(plain, ids.ctypes.data, 3)",
    "dense_size": "L.tf_paged_mla_workspace_bytes(plain, 1, 512, 64, n1)",
    "plan": "L.tf_paged_mla_plan_info(1, 512, 64, n1, 0, 0, ctypes.byref(info), None, None)",
    "dense": "L.tf_paged_mla_attend(plain, 0, BASE, 4, n1, 1, 512, 64, BASE, 0.1, BASE, None, BASE, W, None)",
    "static": "L.tf_paged_mla_attend_static(plain, 0, BASE, 4, n1, 1, 512, 64, BASE, 0.1, BASE, None, None)",
    "dense_fp8_invariant": "L.tf_paged_mla_attend(inv8, 0, BASE, 4, n1, 1, 2, 64, BASE, 0.1, BASE, None, BASE, W, None)",
    "blocks_size": "L.tf_paged_mla_blocks_workspace_bytes(f8, 1, 512, 64, n1, 32)",
    "blocks": "L.tf_paged_mla_attend_blocks(f8, 0, BASE, 4, n1, BASE, 32, 1, 512, 64, BASE, 0.1, BASE, None, BASE, W, None)",
    "shared_size": "L.tf_paged_mla_shared_workspace_bytes(f8, 2, 1, 64, n2, g.ctypes.data, 1, f)",
    "shared": "L.tf_paged_mla_attend_shared(f8, 0, BASE, 4, n2, g.ctypes.data, 1, f, 2, 1, 64, BASE, 0.1, BASE, None, BASE, W, None)",
}


@pytest.fixture(scope="module")
def preload(tmp_path_factory):
    BUILD.build()
    d = tmp_path_factory.mktemp("new")
    src, lib = d / "new.cpp", d / "libnew.so"
    src.write_text(FAIL_NEW)
    subprocess.run([shutil.which("g++") or "g++", "-std=c++17", "-O1", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    return str(lib)


def run(code, lib):
    env = dict(os.environ, LD_PRELOAD=lib, FAIL_NEW=lib, PYTHONPATH=ROOT)
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, timeout=300, cwd=ROOT)


@pytest.mark.parametrize("call", CALLS)
def test_no_exception_leaves_a_call(preload, call):
    code = HOST + f"fail(0)\nrc = {CALLS[call]}\nfail(1 << 63)\nprint('rc', rc, B.TF_E_NOMEM)\n"
    r = run(code, preload)
    assert r.returncode == 0, r.stderr[-500:]
    rc, nomem = map(int, r.stdout.split()[1:])
    assert rc == (0 if call.endswith("size") else nomem)


GPU = """
import ctypes, os, threading
import torch
from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import synth as Y
from paged_mla_kv_gb300.harness import Resident
fail = ctypes.CDLL(os.environ["FAIL_NEW"]).fail_new
fail.argtypes = [ctypes.c_size_t]
w = Y.custom("oom", 1, lens=[2048], R=1, H=16)
res = Resident(w)
q, L, lens = res.q(), B.lib(), res.lens
out = torch.zeros((1, 1, 16, 512), dtype=torch.bfloat16, device="cuda")
bk = torch.zeros((res.pool.num_pages, 8, 576), dtype=torch.bfloat16, device="cuda")
x = torch.zeros((1, 32), device="cuda")
blk = torch.zeros((1, 1, 4), dtype=torch.int32, device="cuda")
ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
n, st = lens.ctypes.data, torch.cuda.current_stream().cuda_stream
p, pt, mp = res.pool.handle, res.pt.data_ptr(), res.max_pages
calls = [
    lambda: L.tf_paged_mla_attend(p, 0, pt, mp, n, 1, 1, 16, q.data_ptr(), 0.1, out.data_ptr(), None, ws.data_ptr(), 1 << 26, st),
    lambda: L.tf_block_scores(p, bk.data_ptr(), pt, mp, n, 1, 1, 16, q.data_ptr(), None, 0.1, 1, 1, x.data_ptr(), 32, None, st),
    lambda: L.tf_paged_mla_attend_blocks(p, 0, pt, mp, n, blk.data_ptr(), 4, 1, 1, 16, q.data_ptr(), 0.1, out.data_ptr(), None,
                                         ws.data_ptr(), 1 << 26, st)]
assert [c() for c in calls] == [0, 0, 0]
got = []
zero = (ctypes.c_int64 * 1)(0)
def thread():                       # its parameter blocks are not made yet; the runtime's own are after the first call
    got.append(L.tf_block_keys_update(p, 0, pt, mp, zero, n, 1, bk.data_ptr(), st))
    for c in calls:
        fail(4096)
        rc = c()
        fail(1 << 63)
        got.append(rc)
    got.extend(c() for c in calls)
t = threading.Thread(target=thread)
t.start(); t.join()
torch.cuda.synchronize()
print("rc", *got)
"""


@pytest.mark.gpu
def test_no_exception_leaves_a_launch(preload):
    r = run(GPU, preload)
    assert r.returncode == 0, r.stderr[-1000:]
    assert list(map(int, r.stdout.split()[1:])) == [0] + [B.TF_E_NOMEM] * 3 + [0] * 3
