"""Page tables with entries that a call has no use for: they are not looked at, whatever the batch's size and
the pool's format."""
import numpy as np
import pytest
import torch

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from paged_mla_kv_gb300 import synth as Y
from paged_mla_kv_gb300.harness import Resident
from tests.gpu_common import bits, no_device_error
from tests.test_gpu_blocks import run_blocks, run_shared, shared_workload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()
    B.lib()


# 16 pages a stream; 64 query rows of a stream over 32 blocks each: the rows of an FP8 pool are expanded to BF16
# pages first.  2 rows: they are not.
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("R", [2, 64])
@pytest.mark.parametrize("gone", ["below", "past", "far"])
def test_unlisted_pages_may_be_gone(R, fp8, gone):
    w = Y.custom("gone", 180, lens=[8192, 8192], R=R, H=64, q_std=1.0, value_std=0.5)
    res = Resident(w, fp8=fp8)
    g = np.random.default_rng(4)
    use = np.array([b for b in range(128) if b // 8 not in (3, 4, 11)])    # these pages are given back
    blk = np.stack([[np.concatenate([[127], g.permutation(use[:-1])[:31]]) for _ in range(R)] for _ in range(2)])
    blk = torch.from_numpy(blk.astype(np.int32)).cuda()
    good = run_blocks(res, w, blk)
    no_device_error(res.pool)
    kept = res.pt
    n = res.pool.num_pages
    # "past": ids behind the pool that would be pages of the expanded rows, if there are more of those
    ids = {"below": [-1, -5, -2 ** 31], "past": [n, n + 1, n + 2], "far": [2 ** 31 - 1, 2 ** 30, n]}[gone]
    res.pt = kept.clone()
    for s in range(2):
        res.pt[s, [3, 4, 11]] = torch.tensor(ids, dtype=torch.int32, device="cuda")
    out, lse = run_blocks(res, w, blk)
    no_device_error(res.pool)
    assert np.array_equal(bits(out), bits(good[0])) and torch.equal(lse, good[1])
    # one entry that a list names is recorded by its own id
    res.pt[1, 11] = kept[1, 11]
    res.pt[0, 5] = ids[0]
    blk[:, :, 5] = 42
    run_blocks(res, w, blk)
    assert res.pool.last_error() == (B.TF_E_DEVICE, ids[0])
    res.pt = kept
    run_blocks(res, w, blk)
    no_device_error(res.pool)


def test_bad_ids_between_the_pools_pages_and_the_expanded_ones():
    """Streams that share pages: the expanded rows are more pages than the pool has."""
    w = Y.custom("goneshare", 181, lens=[4096] * 6, R=64, H=64, share=[(0, 0)] + [(0, 7)] * 5, q_std=1.0, value_std=0.5)
    res = Resident(w, fp8=True)
    n = res.pool.num_pages
    assert n < 6 * 8 - 4
    blk = torch.arange(32, dtype=torch.int32, device="cuda").expand(6, 64, 32).contiguous()
    good = run_blocks(res, w, blk)
    no_device_error(res.pool)
    kept = res.pt
    res.pt = kept.clone()
    res.pt[:, 5] = n + 3
    out, lse = run_blocks(res, w, blk)      # blocks 40 .. 47 are in no list
    no_device_error(res.pool)
    assert np.array_equal(bits(out), bits(good[0])) and torch.equal(lse, good[1])
    res.pt = kept.clone()
    res.pt[4, 2] = n + 3
    run_blocks(res, w, blk)
    assert res.pool.last_error() == (B.TF_E_DEVICE, n + 3)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H", [64, 16])
def test_shared_pages_without_own_rows_may_be_gone(H, fp8):
    """A prefix that ends inside a page and streams that hold nothing behind it: their own entry of that page is not
    needed, no more than those of the pages before it."""
    S, prefix = (16, 20 * 512 + 64) if H == 64 else (64, 40 * 512 + 64)
    w, sizes, prefixes = shared_workload("shgone", 182, [(prefix, [0] * S)], 1, H)
    res = Resident(w, fp8=fp8)
    good = run_shared(res, w, sizes, prefixes)
    no_device_error(res.pool)
    res.pt = res.pt.clone()
    res.pt[1:, :] = -1
    out, lse = run_shared(res, w, sizes, prefixes)
    no_device_error(res.pool)
    assert np.array_equal(bits(out), bits(good[0])) and torch.equal(lse, good[1])
    res.pt[0, 3] = -9
    run_shared(res, w, sizes, prefixes)
    assert res.pool.last_error() == (B.TF_E_DEVICE, -9)


def test_dense_attention_of_expanded_rows_records_a_bad_page():
    """A batch-invariant FP8 pool: every row is expanded first, and every page is read."""
    w = Y.custom("goned", 183, lens=[3000, 700], R=1, H=16)
    res = Resident(w, fp8=True, invariant=True)
    good = res.attend(res.q())
    no_device_error(res.pool)
    kept = res.pt
    for at, bad in (((0, 2), -3), ((1, 1), res.pool.num_pages), ((0, 5), 1 << 30)):
        res.pt = kept.clone()
        res.pt[at] = bad
        res.attend(res.q())
        assert res.pool.last_error() == (B.TF_E_DEVICE, bad)
    res.pt = kept
    again = res.attend(res.q())
    no_device_error(res.pool)
    assert np.array_equal(bits(good[0]), bits(again[0]))
