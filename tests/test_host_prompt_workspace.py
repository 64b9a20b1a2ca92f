"""A workspace tensor is memory in one piece: the call writes nbytes behind its first value.  No GPU."""
import pytest
import torch

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from tests.test_host_block_devices import On
from tests.test_host_prompt import calls


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()
    B.lib()


@pytest.mark.parametrize("ws", [torch.zeros(1, dtype=torch.uint8).expand(4096), torch.zeros(8192, dtype=torch.uint8)[::2],
                                torch.zeros(64, 128, dtype=torch.uint8)[:, :64]])
def test_pieces_are_refused(ws):
    f, ts = calls()["attend"]
    with pytest.raises(B.TFError) as e:
        f({k: On(ws if k == "ws" else v, 0) for k, v in ts.items()})
    assert e.value.code == B.TF_E_ARG and "form" in str(e.value)
