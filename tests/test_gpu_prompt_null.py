"""Attention of prompts without keys: null pointers for keys and values, zeros and -inf out."""
import ctypes

import pytest
import torch

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from tests.gpu_common import no_device_error

pytestmark = pytest.mark.gpu


def test_null_keys_and_values():
    BUILD.build()
    pool = B.KVPool(1, 1)
    q = torch.randn(300, 4, 128, device="cuda").bfloat16()
    out, lse = torch.full_like(q, float("nan")), torch.full((300, 4), float("nan"), device="cuda")
    view = lambda t: ctypes.byref(B.tf_heads(t.data_ptr(), t.stride(0), t.stride(1)))
    n, m = (ctypes.c_int64 * 2)(299, 1), (ctypes.c_int64 * 2)(0, 0)
    rc = B.lib().tf_prompt_attend(pool.handle, n, m, 2, 4, 2, 128, 128, view(q), None, None, 0, None, 0.1, 1, view(out), lse.data_ptr(), None, 0,
                                  torch.cuda.current_stream().cuda_stream)
    assert rc == B.TF_OK
    no_device_error(pool)
    assert not out.any() and torch.isneginf(lse).all()
