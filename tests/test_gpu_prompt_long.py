"""Attention over very long streams: the sums keep their value.

Keys and values overlap (rows eight values apart), so that a million of them fit anywhere.  Tolerance, with u = 2^-8 half
a bf16 step: the weights' rounding u, the output's u |ref|, and 2^-9 for the tensor cores' sums over a part of 131,072
keys (8,192 product steps, each cut by 2^-22 at most).  A score of up to 192 products is off by scale 193 2^-23 sum|q k|, below
2^-11 for normal values (a sum of 192 such magnitudes is about 122, the scale 0.072); an output by twice that, lse by it once.
"""
import pytest
import torch

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from tests.gpu_common import no_device_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()
    B.lib()


def overlapping(n, dim, g, positive):
    x = torch.rand(n * 8 + dim, generator=g, device="cuda") + 0.5 if positive else torch.randn(n * 8 + dim, generator=g, device="cuda")
    return x.bfloat16().as_strided((n, 1, dim), (8, dim, 1))


@pytest.mark.parametrize("dqk,dv", [(64, 64), (192, 128)])
@pytest.mark.parametrize("rows", [1, 300, 152 * 256])
@pytest.mark.parametrize("nk", [131072, 131073, 1 << 20, 3000001])
def test_long_sums(nk, rows, dqk, dv):
    if rows > 300 and dqk > 64 and nk > 1 << 20:
        pytest.skip("half a second of products")
    g = torch.Generator(device="cuda").manual_seed(nk + rows)
    pool = B.KVPool(1, 1)
    k, v = overlapping(nk, dqk, g, False), overlapping(nk, dv, g, True)
    q = torch.randn(rows, 1, dqk, generator=g, device="cuda").bfloat16()
    out, lse = torch.empty(rows, 1, dv, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, 1, device="cuda")
    n = B.tf_prompt_workspace_bytes([rows], [nk], 1, 1, dqk, dv, causal=False)
    B.tf_prompt_attend(pool, [rows], [nk], q, k, v, dqk ** -0.5, out, lse=lse, causal=False,
                       ws=torch.empty(n, dtype=torch.uint8, device="cuda") if n else None)
    no_device_error(pool)
    some = sorted({0, rows // 2, rows - 1})
    qs = q[some, 0].double() * dqk ** -0.5
    num, den = torch.zeros(len(some), dv, dtype=torch.float64, device="cuda"), torch.zeros(len(some), 1, dtype=torch.float64, device="cuda")
    for a in range(0, nk, 1 << 17):
        b = min(nk, a + (1 << 17))
        p = torch.exp(qs @ k[a:b, 0].double().T)
        num += p @ v[a:b, 0].double()
        den += p.sum(1, keepdim=True)
    ref = num / den                                   # of positive values: its own sum of magnitudes
    assert ((out[some, 0].double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -9 + 2.0 ** -10 + 2.0 ** -8) * ref).all()
    # rounding to nearest evens out; the drift of a cut sum does not
    assert abs(((out[some, 0].double() - ref) / ref).mean().item()) <= 2.0 ** -9 + 2.0 ** -12
    assert (lse[some, 0].double() - den[:, 0].log()).abs().max().item() <= 2.0 ** -11
