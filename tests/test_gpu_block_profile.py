"""Launch timing of the block calls."""
import pytest
import torch

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from paged_mla_kv_gb300 import synth as Y
from paged_mla_kv_gb300.harness import Resident

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
def test_block_keys_and_scores_are_timed(fp8):
    BUILD.build()
    w = Y.custom("prof", 190, lens=[2000, 300], R=1, H=16)
    res = Resident(w, fp8=fp8)
    bk = torch.zeros((res.pool.num_pages, 8, 576), dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((2, 32), device="cuda")

    def step():
        B.tf_block_keys_update(res.pool, 0, res.pt, res.max_pages, [0, 0], w.lens, bk)
        B.tf_block_scores(res.pool, bk, res.pt, res.max_pages, w.lens, res.q(), w.scale, x)

    step()
    res.pool.profile(True)
    for _ in range(3):
        step()
    B.tf_block_keys_update(res.pool, 0, res.pt, res.max_pages, w.lens, w.lens, bk)   # no new rows: no launch
    res.pool.profile(False)
    step()
    for kind in (B.PROF_BLOCK_KEYS, B.PROF_BLOCK_SCORES):
        ms, n = res.pool.profile_read(kind)
        assert n == 3 and 0 < ms < 100
        assert res.pool.profile_read(kind) == (0.0, 0)
    assert [res.pool.profile_read(k)[1] for k in range(5)] == [0] * 5
    with pytest.raises(B.TFError):
        res.pool.profile_read(7)
