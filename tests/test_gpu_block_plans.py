"""Each way that attention over listed blocks deals out and merges its work, with the plan asserted, so that no
case slides to another path: clusters of 2 (half of the columns stay in shared memory), larger ones, clusters of
several head groups, and even cuts without a cluster (partials that begin and end inside a CTA's run)."""
import numpy as np
import pytest
import torch

from oracle import blocks as K
from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from paged_mla_kv_gb300 import synth as Y
from paged_mla_kv_gb300.harness import Resident
from tests.gpu_common import bits, no_device_error
from tests.test_gpu_blocks import check_blocks, check_row, host, random_lists, rows64, run_blocks, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()
    B.lib()


def run_twice(res, w, blk):
    out, lse = run_blocks(res, w, blk)
    no_device_error(res.pool)
    again = run_blocks(res, w, blk)
    assert np.array_equal(bits(out), bits(again[0])) and torch.equal(lse, again[1])
    return out, lse


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("S,H", [(64, 64), (62, 40), (60, 33), (64, 32), (64, 17), (32, 128)])
def test_clusters_of_two(S, H, fp8):
    g = np.random.default_rng(H)
    lens = g.integers(2050, 3000, S).tolist()
    lens[1], lens[2], lens[3] = 1, 64, 130       # units of one, one and three tiles: a CTA without one
    w = Y.custom("two", 200 + H, lens=lens, R=1, H=H, q_std=1.0, value_std=0.5)
    p = B.tf_paged_mla_blocks_plan_info(S, 1, H, lens, 32)
    assert p["merge"] == 2, p
    res = Resident(w, fp8=fp8)
    blk = random_lists(w, 32, H)
    blk[4] = -1                                  # no key at all
    blk[5, :, 16:] = -1                          # nor in the second CTA's half
    out, lse = run_twice(res, w, blk)
    check_blocks(res, w, blk, out, lse, fp8)
    assert torch.isneginf(lse[4]).all() and not out[4].any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("S,H,k,merge", [
    (3, 96, 3, 3), (12, 96, 7, 4), (14, 128, 8, 4), (8, 96, 10, 5), (8, 128, 9, 5), (5, 16, 5, 5), (6, 96, 6, 6), (5, 96, 7, 7),
    (1, 100, 7, 7), (1, 16, 8, 8), (4, 96, 8, 8), (2, 128, 8, 8)])
def test_larger_clusters(S, H, k, merge, fp8):
    lens = [64 * k + 100 + 37 * s for s in range(S)]
    if S > 2:
        lens[1] = 65                             # two tiles: CTAs without one
    w = Y.custom("more", 210 + H + k, lens=lens, R=1, H=H, q_std=1.0, value_std=0.5)
    p = B.tf_paged_mla_blocks_plan_info(S, 1, H, lens, k)
    assert p["merge"] == merge, p
    res = Resident(w, fp8=fp8)
    blk = random_lists(w, k, k)
    out, lse = run_twice(res, w, blk)
    check_blocks(res, w, blk, out, lse, fp8)


@pytest.mark.parametrize("S,R,H,n,k,fp8", [
    (1, 2000, 16, 6000, 32, False), (1, 1000, 64, 9000, 40, False), (1, 700, 96, 5000, 21, False), (2, 40, 16, 20000, 32, False),
    (1, 2000, 16, 6000, 32, True),       # the rows are expanded first
    (2, 40, 16, 20000, 32, True), (3, 27, 80, 30000, 30, True)])
def test_even_cuts(S, R, H, n, k, fp8):
    w = Y.custom("even", 220 + R + H, lens=[n - 77 * s for s in range(S)], R=R, H=H, q_std=1.0, value_std=0.5)
    p = B.tf_paged_mla_blocks_plan_info(S, R, H, w.lens, k)
    b = [(int(x) >> 32, int(x) & 0xffffffff) for x in p["bounds"]]
    assert not p["merge"] and p["cut"], p
    # CTAs that begin and end inside a unit, of which the second partial has the CTA's other slot
    both = [i for i in range(p["ctas"]) if b[i][1] and b[i + 1][1] and b[i][0] != b[i + 1][0]]
    assert both, p
    res = Resident(w, fp8=fp8)
    blk = random_lists(w, k, R)
    out, lse = run_twice(res, w, blk)
    hg = -(-H // 64)
    units = {u for u, t in b[:-1] if t}                                   # the cut ones
    units |= {u + 1 for u in units} | {u - 1 for u in units} | {0, S * R * hg - 1}
    rows = sorted({u // hg for u in units if 0 <= u < S * R * hg})
    rows = rows[::max(1, len(rows) // 120)] + rows[-1:]
    o, l, q, lst = host(out), host(lse), values(w.q(0)), blk.cpu().numpy()
    held = [rows64(w, s, fp8) for s in range(S)]
    for x in rows:
        s, r = divmod(x, R)
        pos = int(w.lens[s]) - R + r
        check_row(o[s, r], l[s, r], q[s, r], *held[s], K.rows_of_list(lst[s, r][:min(k, pos // 64 + 1)].tolist(), pos), w.scale)


def test_a_plan_query_is_the_calls_plan():
    """The workspace's size and the SMs of this device, not of another."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    a = B.tf_paged_mla_blocks_plan_info(300, 1, 64, [4000] * 300, 60)
    b = B.tf_paged_mla_blocks_plan_info(300, 1, 64, [4000] * 300, 60, sms)
    assert a["ctas"] == b["ctas"] <= sms and np.array_equal(a["bounds"], b["bounds"])
