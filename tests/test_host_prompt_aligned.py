"""Pointers to 4-byte values that are not on 4 bytes are refused: a kernel's access there would fault.  No GPU."""
import ctypes

import pytest

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from tests.test_host_prompt import BASE, _pool, heads, i64


@pytest.fixture(scope="module", autouse=True)
def L():
    BUILD.build()
    return B.lib()


@pytest.mark.parametrize("off", [1, 2, 3, 5, 15])
def test_page_tables(L, off):
    assert L.tf_paged_append_rope(_pool(), 0, BASE + off, 4, i64(0), i64(5), 1, BASE, 576, None, 0.0, None, None) == B.TF_E_ARG
    assert L.tf_paged_read(_pool(), 0, BASE + off, 4, i64(0), i64(5), 1, BASE, 512, None, 0, None) == B.TF_E_ARG


@pytest.mark.parametrize("off", [1, 2, 3, 5, 15])
def test_sums(L, off):
    h = heads()
    assert L.tf_prompt_attend(_pool(), i64(3), i64(3), 1, 4, 4, 128, 128, h, h, None, 0, h, 0.1, 1, h, BASE + off, None, 0, None) == B.TF_E_ARG
