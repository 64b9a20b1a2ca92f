"""Block keys of a stream that goes on from a kept state: the rows are copied to fresh pages, whose keys are then
averaged from row 0 (or taken over page by page), and the step behind it chooses what the kept stream would."""
import numpy as np
import pytest
import torch

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from paged_mla_kv_gb300 import synth as Y
from paged_mla_kv_gb300.harness import Resident
from tests.gpu_common import bits, no_device_error
from tests.test_gpu_blocks import run_blocks, run_scores

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()
    B.lib()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 64, 1000, 1536, 3001])
def test_a_resumed_stream_scores_as_the_kept_one(n, fp8):
    w = Y.custom("resume", 230, lens=[n], R=1, H=16, q_std=1.0, value_std=0.5)
    res = Resident(w, fp8=fp8, extra_pages=w.max_pages + 3)
    pages, blocks = -(-n // 512), -(-n // 64)
    left = float("nan")                           # what earlier owners of the pages left
    bk = torch.full((res.pool.num_pages, 8, 576), left, dtype=torch.bfloat16, device="cuda")
    B.tf_block_keys_update(res.pool, 0, res.pt, res.max_pages, [0], [n], bk)
    q = res.q()
    k = min(12, blocks)
    blk = torch.arange(blocks - k, blocks, dtype=torch.int32, device="cuda").view(1, 1, k)

    def step():
        x, _, cols = run_scores(res, w, bk, q, local=2)
        return x[:, :cols], run_blocks(res, w, blk)

    want = step()
    old = res.pt.clone()
    keys = [bk[int(old[0, b // 8]), b % 8].clone() for b in range(blocks)]
    fresh = torch.zeros_like(old)
    fresh[0, :pages] = torch.from_numpy(res.pool.take(pages)).cuda()
    assert not set(fresh[0, :pages].tolist()) & set(old[0, :pages].tolist())
    B.tf_state_copy_rows(res.pool, 0, old[0], fresh[0], n)
    bk[old[0, :pages].long()] = left              # the kept state's pages go back to the pool
    res.pt = fresh
    B.tf_block_keys_update(res.pool, 0, res.pt, res.max_pages, [0], [n], bk)
    for b in range(blocks):
        assert torch.equal(bk[int(fresh[0, b // 8]), b % 8], keys[b])
    got = step()
    no_device_error(res.pool)
    assert torch.equal(got[0], want[0])
    assert np.array_equal(bits(got[1][0]), bits(want[1][0])) and torch.equal(got[1][1], want[1][1])
    # without the averaging the scores say so instead of ranking what the pages held before
    bk[fresh[0, :pages].long()] = left
    x, _, cols = run_scores(res, w, bk, q, local=2)
    free = x[0, 1:max(1, cols - 2)]
    assert torch.isnan(free).all()
