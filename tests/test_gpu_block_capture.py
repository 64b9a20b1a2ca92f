"""Calls that nothing warmed up: the first one of a process made under capture, and two threads that use one FP8
pool at once with workspaces of their own."""
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from paged_mla_kv_gb300 import synth as Y
from paged_mla_kv_gb300.harness import Resident
from tests.gpu_common import bits, no_device_error
from tests.test_gpu_blocks import random_lists, run_blocks, run_shared, shared_workload

pytestmark = pytest.mark.gpu

CAPTURE = """
import sys
import torch
from paged_mla_kv_gb300 import binding as B, synth as Y
from paged_mla_kv_gb300.harness import Resident

S, R, H, n, fp8 = {args}
w = Y.custom("cap", 240, lens=[n] * S, R=R, H=H, q_std=1.0, value_std=0.5)
res = Resident(w, fp8=fp8)                       # appends: the pool has had a launch
q = res.q()
z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
cols, k = -(-n // 64), 8
bk, sc = z(res.pool.num_pages, 8, 576, dt=torch.bfloat16), z(S * R, -(-cols // 4) * 4)
nb, idx, val = z(S * R, dt=torch.int32), z(S * R, k, dt=torch.int32), z(S * R, k)
out, lse, out2, lse2 = z(S, R, H, 512, dt=torch.bfloat16), z(S, R, H), z(S, R, H, 512, dt=torch.bfloat16), z(S, R, H)
ws = z(max(256, B.tf_paged_mla_blocks_workspace_bytes(res.pool, S, R, H, w.lens, k)), dt=torch.uint8)
ws2 = z(max(256, B.tf_paged_mla_shared_workspace_bytes(res.pool, S, R, H, w.lens, [1] * S, [0] * S)), dt=torch.uint8)
wk = z(max(256, B.tf_topk_workspace_bytes(S * R, cols, k)), dt=torch.uint8)

def step():
    B.tf_block_keys_update(res.pool, 0, res.pt, res.max_pages, [0] * S, w.lens, bk)
    B.tf_block_scores(res.pool, bk, res.pt, res.max_pages, w.lens, q, w.scale, sc, nblk=nb, local=2)
    B.tf_topk_blocked(sc, k, idx, val, lens=nb, n=cols, ws=wk)
    B.tf_paged_mla_attend_blocks(res.pool, 0, res.pt, res.max_pages, w.lens, idx, q, w.scale, out, lse, ws)
    B.tf_paged_mla_attend_shared(res.pool, 0, res.pt, res.max_pages, w.lens, [1] * S, [0] * S, q, w.scale, out2, lse2, ws2)

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
all_ = (bk, sc, nb, idx, out, lse, out2, lse2)
assert not any(t.any() for t in all_)            # recorded, not run
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in all_]
for t in all_:
    t.zero_()
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, all_)) and out.any() and out2.any()
assert res.pool.last_error()[0] == 0
print("same")
"""


@pytest.mark.parametrize("args", ["2, 1, 16, 3000, False", "1, 200, 64, 3000, True"])
def test_first_call_of_a_process_is_captured(args):
    BUILD.build()
    r = subprocess.run([sys.executable, "-c", CAPTURE.format(args=args)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


def test_two_threads_on_one_fp8_pool():
    """Calls whose rows are expanded first, from two host threads on two streams."""
    w, sizes, prefixes = shared_workload("thr", 241, [(4096, [40, 70, 600, 45])], 40, 64)
    res = Resident(w, fp8=True)
    blk = random_lists(w, 30, 3)
    want = run_blocks(res, w, blk), run_shared(res, w, sizes, prefixes)
    no_device_error(res.pool)
    got, errors = [[], []], []

    def go(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got[i].append(run_blocks(res, w, blk) if i == 0 else run_shared(res, w, sizes, prefixes))
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # pragma: no cover
            errors.append(e)

    ts = [threading.Thread(target=go, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors
    torch.cuda.synchronize()
    no_device_error(res.pool)
    for i in range(2):
        for out, lse in got[i]:
            assert np.array_equal(bits(out), bits(want[i][0])) and torch.equal(lse, want[i][1])
