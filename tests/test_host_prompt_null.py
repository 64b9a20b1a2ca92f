"""Attention of prompts without keys, or without rows, takes null pointers for what is not there.  No GPU."""
import pytest
import torch

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from tests.test_host_prompt import _pool, heads, i64


@pytest.fixture(scope="module", autouse=True)
def L():
    BUILD.build()
    return B.lib()


def call(L, nq, nk, q, k, v, out):
    return L.tf_prompt_attend(_pool(), i64(nq), i64(nk), 1, 4, 4, 128, 128, q, k, None, 0, v, 0.1, 1, out, None, None, 0, None)


def test_no_rows(L):
    assert call(L, 0, 5, None, heads(), heads(), None) == B.TF_OK
    assert call(L, 0, 0, None, None, None, None) == B.TF_OK
    assert call(L, 0, 5, None, None, None, None) == B.TF_OK      # nothing is read


def test_rows_need_their_tensors(L):
    assert call(L, 3, 0, None, None, None, heads()) == B.TF_E_ARG
    assert call(L, 3, 0, heads(), None, None, None) == B.TF_E_ARG
    assert call(L, 3, 5, heads(), None, heads(), heads()) == B.TF_E_ARG
    assert call(L, 3, 5, heads(), heads(), None, heads()) == B.TF_E_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="would be launched")
def test_no_keys(L):
    assert call(L, 3, 0, heads(), None, None, heads()) == B.TF_E_CUDA     # past the checks: no GPU here
