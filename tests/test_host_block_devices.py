"""The binding refuses tensors that do not lie on the pool's GPU: their addresses mean nothing to a kernel.
No GPU: the pool stands for one of GPU 0, the tensors are the host's or claim another device."""
import types

import pytest
import torch

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD

BF = dict(dtype=torch.bfloat16)


class On:
    """A host tensor that says it lies on GPU `dev`.  Its address is never read: every call here is refused."""

    def __init__(self, t, dev):
        self.t, self.dev = t, dev

    def get_device(self):
        return self.dev

    @property
    def device(self):
        return torch.device("cuda", self.dev)

    @property
    def is_cuda(self):
        return True

    def __getattr__(self, name):
        return getattr(self.t, name)


def calls():
    """name -> (call, its tensors); every form is right."""
    pool = types.SimpleNamespace(handle=None, num_pages=4, device=0)   # a null handle: nothing can be launched
    i32 = dict(dtype=torch.int32)
    t = {"pt": torch.zeros(2, 2, **i32), "bkeys": torch.zeros(4, 8, 576, **BF), "q": torch.zeros(2, 1, 16, 576, **BF),
         "out": torch.zeros(2, 1, 16, 512, **BF), "lse": torch.zeros(2, 1, 16), "blk": torch.zeros(2, 1, 4, **i32),
         "w": torch.zeros(2, 1, 16), "scores": torch.zeros(2, 4), "nblk": torch.zeros(2, **i32),
         "ws": torch.zeros(1024, dtype=torch.uint8)}
    return {
        "tf_block_keys_update": (lambda a: B.tf_block_keys_update(pool, 0, a["pt"], 2, [0, 0], [64, 64], a["bkeys"], stream=0),
                                 {k: t[k] for k in ("pt", "bkeys")}),
        "tf_block_scores": (lambda a: B.tf_block_scores(pool, a["bkeys"], a["pt"], 2, [64, 64], a["q"], 0.1, a["scores"],
                                                        w=a["w"], nblk=a["nblk"], stream=0),
                            {k: t[k] for k in ("pt", "bkeys", "q", "scores", "w", "nblk")}),
        "tf_paged_mla_attend_blocks": (lambda a: B.tf_paged_mla_attend_blocks(pool, 0, a["pt"], 2, [64, 64], a["blk"], a["q"], 0.1,
                                                                              a["out"], a["lse"], a["ws"], stream=0),
                                       {k: t[k] for k in ("pt", "blk", "q", "out", "lse", "ws")}),
        "tf_paged_mla_attend_shared": (lambda a: B.tf_paged_mla_attend_shared(pool, 0, a["pt"], 2, [64, 64], [2], [0], a["q"], 0.1,
                                                                              a["out"], a["lse"], a["ws"], stream=0),
                                       {k: t[k] for k in ("pt", "q", "out", "lse", "ws")})}


CASES = [(c, t) for c, (_, ts) in calls().items() for t in ts]


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()
    B.lib()


@pytest.mark.parametrize("call,tensor", CASES)
@pytest.mark.parametrize("dev", ["host", 1])
def test_a_tensor_elsewhere_is_refused(call, tensor, dev):
    f, ts = calls()[call]
    args = {k: On(v, 0) for k, v in ts.items()}
    args[tensor] = ts[tensor] if dev == "host" else On(ts[tensor], dev)
    with pytest.raises(B.TFError) as e:
        f(args)
    assert e.value.code == B.TF_E_ARG and "not on the pool's device" in str(e.value)


@pytest.mark.parametrize("call", list(calls()))
def test_tensors_on_the_pools_device_reach_the_library(call):
    f, ts = calls()[call]
    with pytest.raises(B.TFError) as e:      # its own refusal of a null pool
        f({k: On(v, 0) for k, v in ts.items()})
    assert e.value.code == B.TF_E_ARG and "device" not in str(e.value)


@pytest.mark.parametrize("call,tensor", [c for c in CASES if c[1] != "ws"])
def test_a_wrong_form_is_told_from_a_wrong_device(call, tensor):
    f, ts = calls()[call]
    args = {k: On(v, 0) for k, v in ts.items()}
    args[tensor] = On(ts[tensor].to(torch.float64 if tensor != "w" else torch.int64), 0)
    with pytest.raises(B.TFError) as e:
        f(args)
    assert e.value.code == B.TF_E_ARG and "form" in str(e.value)
