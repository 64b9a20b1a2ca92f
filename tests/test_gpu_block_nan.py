"""NaN and infinities through block scores and attention over listed blocks: a value that is not a number
stays one, in the columns that it belongs to and nowhere else.  Tolerances as in test_gpu_blocks."""
import numpy as np
import pytest
import torch

from oracle import blocks as K
from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from paged_mla_kv_gb300 import synth as Y
from paged_mla_kv_gb300.harness import Resident
from tests.gpu_common import no_device_error
from tests.test_gpu_blocks import check_row, host, random_lists, rows64, run_blocks, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()
    B.lib()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("S,H,n,k", [
    (1, 16, 2048, 8),       # a unit on a cluster of several CTAs
    (64, 64, 1500, 32),     # on two, each merging half of the columns
    (3, 96, 1500, 8),       # two head groups a row
    (1, 16, 20000, 300),    # cut, merged by a combine pass
    (300, 16, 600, 2)])     # whole units
def test_nan_queries_give_nan(S, H, n, k, fp8):
    w = Y.custom("nanq", 170 + k, lens=[n] * S, R=1, H=H, q_std=1.0, value_std=0.5)
    res = Resident(w, fp8=fp8)
    q = res.q()
    q[0, 0, 3, 5] = float("nan")
    q[S - 1, 0, H - 1, 570] = float("nan")
    blk = random_lists(w, k, k, holes=False)
    out, lse = run_blocks(res, w, blk, q=q)
    no_device_error(res.pool)
    bad = torch.zeros((S, 1, H), dtype=torch.bool)
    bad[0, 0, 3] = bad[S - 1, 0, H - 1] = True
    assert torch.equal(torch.isnan(lse).cpu(), bad)
    assert torch.isnan(out.cpu()[bad]).all() and torch.isfinite(out.cpu()[~bad].float()).all()
    o, l, b, qs = host(out), host(lse), blk.cpu().numpy(), values(w.q(0))
    for s in {0, S - 1}:
        lat, rope = rows64(w, s, fp8)
        fine = ~bad[s, 0].numpy()
        check_row(o[s, 0][fine], l[s, 0][fine], qs[s, 0][fine], lat, rope, K.rows_of_list(b[s, 0].tolist(), n - 1), w.scale)
