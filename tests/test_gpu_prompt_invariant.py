"""Attention of prompts on a TF_POOL_BATCH_INVARIANT pool: a stream's bits do not hang on the rest of the batch."""
import numpy as np
import pytest
import torch

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from tests.gpu_common import bits
from tests.test_gpu_prompt import call, check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()
    B.lib()


@pytest.fixture(scope="module")
def pool():
    return B.KVPool(1, 1, invariant=True)


@pytest.mark.parametrize("dqk,dv,kr", [(192, 128, True), (128, 128, False), (64, 64, False)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,H,Hkv", [
    ([1, 1, 2], [20000, 700, 9001], 8, 1), ([300, 1, 17, 2000], [6000, 129, 17, 2000], 2, 2), ([5, 0, 260, 3], [5, 9, 12345, 40000], 16, 2),
    ([1, 1, 300], [131073, 1000, 262145], 2, 1), ([300, 140, 9], [77, 0, 3], 6, 2),
])
def test_alone_and_in_a_batch(pool, nq, nk, H, Hkv, causal, dqk, dv, kr):
    q, k, v, rot = make(nq, nk, H, Hkv, dqk, dv, kr, seed=51)
    out, lse = call(pool, nq, nk, q, k, v, kr=rot, causal=causal)
    check(nq, nk, q, k, v, rot, causal, out, lse, rows=3)
    a = b = 0
    for n, m in zip(nq, nk):
        if n:
            one, l1 = call(pool, [n], [m], q[a:a + n], k[b:b + m], v[b:b + m], kr=None if rot is None else rot[b:b + m], causal=causal)
            assert np.array_equal(bits(one), bits(out[a:a + n])) and torch.equal(l1, lse[a:a + n])
        a, b = a + n, b + m
    r = list(range(len(nq)))[::-1]              # another order
    rows = lambda t, c: torch.cat([t[sum(c[:s]):sum(c[:s + 1])] for s in r])
    o2, l2 = call(pool, [nq[s] for s in r], [nk[s] for s in r], rows(q, nq), rows(k, nk), rows(v, nk), kr=None if rot is None else rows(rot, nk), causal=causal)
    assert np.array_equal(bits(o2), bits(rows(out, nq))) and torch.equal(l2, rows(lse, nq))
