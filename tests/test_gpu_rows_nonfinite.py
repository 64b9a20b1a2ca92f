"""Rows that are not finite, written by tf_paged_append_rope to both formats of pages and read back.

What is expected follows from the definition alone.  The norm's factor of a row with a NaN is NaN, and with it every
value; of a row with an infinity it is 0: its finite values become 0 and the infinite ones 0 times infinity.  On FP8
pages amax leaves NaN out, as in tf_paged_append, and a value that is NaN has a code that is.
"""
import numpy as np
import pytest
import torch

from oracle import fp8 as F8
from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from tests.gpu_common import bits, no_device_error
from tests.test_gpu_rows import held, randn, tables

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()
    B.lib()


def rows_of(*special, zeros=False, seed=0):
    """Random rows (or rows of zeros), each with the values of one of `special` at a few places."""
    x = randn(len(special), 576, seed=seed)
    if zeros:
        x[:, :512] = 0
    for i, vals in enumerate(special):
        for k, v in enumerate(vals):
            x[i, (17 + 263 * k + 5 * i) % 512] = v
    return x


SPECIAL = [(NAN,), (INF,), (-INF,), (INF, -INF), (NAN, INF), (-NAN, -INF, NAN), (), (NAN, NAN)]


def write_and_read(x, fp8, gain):
    pool = B.KVPool(1, 2, poison=True, fp8=fp8)
    pt, mp = tables(pool, [x.shape[0]])
    B.tf_paged_append_rope(pool, 0, pt, mp, [0], [x.shape[0]], x, gain=gain, eps=1e-6)
    lat = torch.empty((x.shape[0], 512), dtype=torch.bfloat16, device="cuda")
    B.tf_paged_read(pool, 0, pt, mp, [0], [x.shape[0]], latent=lat)
    no_device_error(pool)
    return lat, pool, int(pt[0, 0])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("zeros", [False, True])
def test_norm_of_rows_that_are_not_finite(fp8, zeros):
    x = rows_of(*SPECIAL, zeros=zeros, seed=1)
    x[6, :512] = NAN                                      # every value
    gain = (1 + 0.25 * torch.randn(512, device="cuda")).bfloat16()
    lat, pool, page = write_and_read(x, fp8, gain)
    for i, row in enumerate(x[:, :512]):
        if torch.isnan(row).any():
            assert torch.isnan(lat[i]).all(), i
        else:
            inf = torch.isinf(row)
            assert inf.any() and torch.isnan(lat[i][inf]).all() and (lat[i][~inf] == 0).all(), i
    if fp8:                                               # the codes say it, whatever the scale
        codes = F8.decode_table()[held(pool)[0][page, :x.shape[0]]]
        assert np.array_equal(np.isnan(codes), torch.isnan(lat).cpu().numpy())


@pytest.mark.parametrize("zeros", [False, True])
def test_a_nan_keeps_its_place_without_a_norm(zeros):
    """FP8: the other values keep theirs; of zeros and NaN too."""
    x = rows_of((NAN,), (-NAN, NAN), (NAN, NAN, NAN), zeros=zeros, seed=2)
    lat, pool, page = write_and_read(x, True, None)
    nan = torch.isnan(x[:, :512])
    assert torch.equal(torch.isnan(lat), nan)
    clean = x[:, :512].float().masked_fill(nan, 0).cpu().numpy()
    want = torch.from_numpy(F8.dequantize_rows(*F8.quantize_rows(clean)).astype(np.float32)).bfloat16().cuda()
    assert torch.equal(lat[~nan], want[~nan])
    bf, _, _ = write_and_read(x, False, None)
    assert np.array_equal(bits(bf), bits(x[:, :512]))


def test_codes_of_infinities_equal_the_appends():
    """Scale infinite: finite values have the code 0, infinite ones and NaN NaN, bit for bit as tf_paged_append has them."""
    x = torch.cat([rows_of((INF,), (-INF,), (INF, -INF), (NAN, INF), (NAN,), (-NAN, NAN), seed=3),
                   rows_of((INF,), (-INF,), (INF, -INF), (NAN, INF), zeros=True, seed=4)])
    x = torch.cat([x, torch.full((1, 576), INF, device="cuda").bfloat16()])
    n = x.shape[0]
    lat, b, page = write_and_read(x, True, None)
    a = B.KVPool(1, 2, poison=True, fp8=True)
    pa, mp = tables(a, [n])
    B.tf_paged_append(a, 0, pa, mp, [0], x[:, :512].contiguous().view(1, n, 512), x[:, 512:].contiguous().view(1, n, 64))
    no_device_error(a)
    for u, v in zip(held(a), held(b)):
        assert np.array_equal(u[int(pa[0, 0]), :n].view(np.uint8), v[page, :n].view(np.uint8))
    assert torch.isnan(lat[torch.isinf(x[:, :512]).any(1)]).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_neighbours_of_such_rows_keep_their_bits(fp8):
    x = randn(64, 576, seed=5)
    gain = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    clean, _, _ = write_and_read(x, fp8, gain)
    y = x.clone()
    y[5], y[6, 3], y[40, 511] = NAN, INF, NAN
    lat, _, _ = write_and_read(y, fp8, gain)
    same = torch.tensor([i not in (5, 6, 40) for i in range(64)])
    assert np.array_equal(bits(lat[same]), bits(clean[same]))
