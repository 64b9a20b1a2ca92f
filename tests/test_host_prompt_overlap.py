"""Outputs that overlap themselves are refused (rows or heads of stride 0, or less than their width apart).  No GPU."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from tests.test_host_block_devices import On
from tests.test_host_prompt import BASE, _pool, heads, i64


@pytest.fixture(scope="module", autouse=True)
def L():
    BUILD.build()
    return B.lib()


def overlaps(rows, row, H, head, width):
    at = sorted(r * row + h * head for r, h in itertools.product(range(rows), range(H)))
    return any(b - a < width for a, b in zip(at, at[1:]))


def cases():
    r = np.random.default_rng(1)
    out = [(5, 0, 2, 64), (5, 256, 2, 0), (5, 256, 2, 32), (5, 64, 3, 64), (3, 64, 2, 192), (4, 64, 2, 192), (3, -64, 2, 192), (4, -64, 2, -192), (5, 1 << 61, 3, 64),
           (2, 1 << 62, 3, 1 << 62), (2, -(1 << 62), 128, 1 << 61), (2 ** 31 - 1, 64, 2, 64 * (2 ** 31 - 1)), (2 ** 31 - 1, 64, 2, 64 * (2 ** 31 - 2))]
    for _ in range(300):
        out.append((int(r.integers(1, 9)), 8 * int(r.integers(-60, 60)), int(r.integers(1, 9)), 8 * int(r.integers(-60, 60))))
    return out


def known(rows, row, H, head, width):
    if rows < 100:
        return overlaps(rows, row, H, head, width)
    return head < rows * row


@pytest.mark.parametrize("case", range(len(cases())))
def test_rotation(L, case):
    """Of the same tensor as it was made, and of others: nothing is launched, as there is no GPU, where it is not refused."""
    rows, row, H, head = cases()[case]
    rope = B.tf_rope_make(64)
    rc = L.tf_rope_apply(ctypes.addressof(rope), i64(0), i64(rows), 1, H, BASE, 0, 0, BASE, row, head, None)
    bad = known(rows, row, H, head, 64)
    if torch.cuda.is_available() and not bad:
        pytest.skip("would be launched")
    assert (rc == B.TF_E_ARG) == bad, (rows, row, H, head, rc)


@pytest.mark.parametrize("case", range(len(cases())))
def test_attention(L, case):
    rows, row, H, head = cases()[case]
    bad = known(rows, row, H, head, 64)
    if torch.cuda.is_available() and not bad:
        pytest.skip("would be launched")
    q = heads(row=8 * 64, head=64)
    rc = L.tf_prompt_attend(_pool(), i64(rows), i64(0), 1, H, H, 64, 64, q, q, None, 0, q, 0.1, 1, heads(row=row, head=head), None, None, 0, None)
    assert (rc == B.TF_E_ARG) == bad, (rows, row, H, head, rc)


def test_expanded_tensors_are_refused():
    pool = type("P", (), dict(handle=_pool(), device=0))()
    bf = dict(dtype=torch.bfloat16)
    q, k, v = torch.zeros(5, 4, 64, **bf), torch.zeros(7, 2, 64, **bf), torch.zeros(7, 2, 64, **bf)
    for out in (torch.zeros(1, 4, 64, **bf).expand(5, 4, 64), torch.zeros(5, 1, 64, **bf).expand(5, 4, 64)):
        with pytest.raises(B.TFError) as e:
            B.tf_prompt_attend(pool, [5], [7], On(q, 0), On(k, 0), On(v, 0), 0.1, On(out, 0), stream=0)
        assert e.value.code == B.TF_E_ARG
        with pytest.raises(B.TFError) as e:
            B.tf_rope_apply(B.tf_rope_make(64), [0], [5], On(q, 0), On(out, 0), stream=0)
        assert e.value.code == B.TF_E_ARG
