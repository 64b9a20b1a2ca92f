"""The work plan of attention over very long streams: no item goes over more than 131,072 keys."""
import numpy as np
import pytest

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()
    B.lib()


@pytest.mark.parametrize("sms", [1, 152, 240])
@pytest.mark.parametrize("nq,nk", [([152 * 256], [1 << 20]), ([100000], [100000]), ([100000], [131072]), ([100000], [131073]),
                                   ([3, 70000, 1], [500000, 200000, 5]), ([1], [2 ** 31 - 1]), ([256], [1 << 28])])
@pytest.mark.parametrize("causal", [True, False])
def test_parts_of_a_long_stream(nq, nk, sms, causal):
    p = B.tf_prompt_plan_info(nq, nk, 1, 1, 64, 64, causal=causal, sms=sms)
    most = max(-(-k // 128) for n, k in zip(nq, nk) if n)
    assert p["splits"] >= -(-most // 1024)
    assert (p["slots"] > 0) == (p["splits"] > 1)


def test_the_workspace_of_a_long_stream_is_asked_for():
    assert B.tf_prompt_workspace_bytes([100000], [131072], 64, 64, 192, 128) == 0
    n = B.tf_prompt_workspace_bytes([100000], [131073], 64, 64, 192, 128)
    assert n >= 2 * 100000 * 64 * (128 * 4 + 8)


def test_plans_of_streams_that_are_not_long_stay():
    """Up to 131,072 keys nothing changes where whole items fill the SMs."""
    r = np.random.default_rng(3)
    for _ in range(50):
        nk = [int(x) for x in r.integers(1, 131073, 8)]
        assert B.tf_prompt_plan_info(nk, nk, 64, 64, 192, 128, sms=152)["splits"] == 1
