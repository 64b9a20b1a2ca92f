"""Host side of the block and shared-prefix calls: what they refuse before any launch, their workspace
sizes, and the header.  No GPU: the pool is made over an address that is never read."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 1 << 40


@pytest.fixture(scope="module")
def L():
    BUILD.build()
    return B.lib()


def _pool(pages=32, caches=2, fp8=False):
    d = B.make_desc(caches, pages, fp8=fp8)
    h = ctypes.c_void_p()
    assert B.lib().tf_kvpool_create(ctypes.byref(d), ctypes.c_void_p(BASE), B.tf_kvpool_bytes(d), ctypes.byref(h)) == 0
    return h


def _arr(a, t):
    a = np.asarray(a, t)
    return a, a.ctypes.data


@pytest.mark.parametrize("fp8", [False, True])
def test_block_keys_refusals(L, fp8):
    h = _pool(fp8=fp8)
    assert L.tf_block_keys_bytes(h) == 32 * 8 * 576 * 2 and L.tf_block_keys_bytes(None) == 0
    keep = []

    def call(pool=h, cache=0, pt=BASE, mp=4, start=(0, 5), lens=(100, 2048), S=2, bk=BASE):
        f, pf = _arr(start, np.int64)
        n, pn = _arr(lens, np.int64)
        keep.extend([f, n])
        return L.tf_block_keys_update(pool, cache, pt, mp, pf, pn, S, bk, None)

    assert call(pool=None) == B.TF_E_ARG
    assert call(bk=None) == B.TF_E_ARG and call(bk=BASE + 8) == B.TF_E_ARG
    assert call(S=0) == B.TF_E_ARG and call(S=513) == B.TF_E_ARG and call(mp=0) == B.TF_E_ARG
    assert call(cache=2) == B.TF_E_RANGE and call(cache=-1) == B.TF_E_RANGE
    assert call(pt=None, mp=17) == B.TF_E_RANGE                  # 34 window pages, 32 in the pool
    assert call(start=(-1, 0)) == B.TF_E_RANGE and call(start=(101, 0)) == B.TF_E_RANGE
    assert call(lens=(100, 2049)) == B.TF_E_RANGE
    assert call(mp=1 << 30, lens=(100, 1 << 31)) == B.TF_E_UNSUPPORTED
    assert call(start=(100, 2048)) == B.TF_OK                    # no new rows: nothing is launched
    assert call(start=(0, 0), lens=(0, 0)) == B.TF_OK
    n, pn = _arr([1], np.int64)
    assert L.tf_block_keys_update(h, 0, BASE, 4, None, pn, 1, BASE, None) == B.TF_E_ARG
    assert L.tf_block_keys_update(h, 0, BASE, 4, pn, None, 1, BASE, None) == B.TF_E_ARG


def test_block_scores_refusals(L):
    h = _pool()
    keep = []

    def call(pool=h, bk=BASE, pt=BASE, mp=4, lens=(100, 2048), S=2, R=2, H=16, q=BASE, w=None, scale=0.1, sink=1,
             local=1, out=BASE, ld=32):
        n, pn = _arr(lens, np.int64)
        keep.append(n)
        return L.tf_block_scores(pool, bk, pt, mp, pn, S, R, H, q, w, scale, sink, local, out, ld, None, None)

    for bad in ({"pool": None}, {"bk": None}, {"bk": BASE + 2}, {"q": None}, {"q": BASE + 8}, {"out": None},
                {"out": BASE + 4}, {"S": 0}, {"R": 0}, {"H": 0}, {"H": 129}, {"mp": 0}, {"scale": 0.0},
                {"scale": float("nan")}, {"scale": float("inf")}, {"sink": -1}, {"local": 0}, {"ld": 31}, {"ld": 28}):
        assert call(**bad) == B.TF_E_ARG, bad
    for bad in ({"lens": (1, 2048)}, {"lens": (100, 2049)}, {"pt": None, "mp": 17}):
        assert call(**bad) == B.TF_E_RANGE, bad
    assert call(R=1 << 24, H=128, lens=(1 << 25, 1 << 25), mp=1 << 20) == B.TF_E_UNSUPPORTED
    assert call(lens=(100, 1 << 31), mp=1 << 30, ld=1 << 30) == B.TF_E_UNSUPPORTED


@pytest.mark.parametrize("fp8", [False, True])
def test_attend_blocks_refusals(L, fp8):
    h = _pool(fp8=fp8)
    keep = []

    def call(pool=h, cache=0, pt=BASE, mp=4, lens=(100, 2048), blk=BASE, k=32, S=2, R=2, H=16, q=BASE, scale=0.1,
             out=BASE, ws=BASE, n=1 << 40):
        a, p = _arr(lens, np.int64)
        keep.append(a)
        return L.tf_paged_mla_attend_blocks(pool, cache, pt, mp, p, blk, k, S, R, H, q, scale, out, None, ws, n, None)

    need = B.tf_paged_mla_blocks_workspace_bytes(None, 2, 2, 16, [100, 2048], 32)
    assert need > 0
    for bad in ({"pool": None}, {"blk": None}, {"k": 0}, {"k": -1}, {"S": 0}, {"S": 513}, {"R": 0}, {"H": 129}, {"mp": 0},
                {"q": None}, {"q": BASE + 2}, {"out": None}, {"out": BASE + 8}, {"scale": -1.0}, {"scale": float("inf")},
                {"ws": None}, {"ws": BASE + 128}):
        assert call(**bad) == B.TF_E_ARG, bad
    for bad in ({"cache": 2}, {"lens": (1, 2048)}, {"lens": (100, 2049)}, {"pt": None, "mp": 17}):
        assert call(**bad) == B.TF_E_RANGE, bad
    assert call(n=need - 1) == B.TF_E_NOMEM
    assert call(R=1 << 24, H=128, lens=(1 << 25, 1 << 25), mp=1 << 20) == B.TF_E_UNSUPPORTED
    assert call(lens=(100, 1 << 31), mp=1 << 30) == B.TF_E_UNSUPPORTED


@pytest.mark.parametrize("fp8", [False, True])
def test_attend_shared_refusals(L, fp8):
    h = _pool(fp8=fp8)
    keep = []

    def call(pool=h, cache=0, pt=BASE, mp=4, lens=(1000, 2048, 30), g=(2, 1), G=2, f=(640, 0), S=3, R=2, H=16, q=BASE,
             scale=0.1, out=BASE, ws=BASE, n=1 << 40):
        a, p = _arr(lens, np.int64)
        b, pb = _arr(g, np.int32)
        c, pc = _arr(f, np.int64)
        keep.extend([a, b, c])
        return L.tf_paged_mla_attend_shared(pool, cache, pt, mp, p, pb, G, pc, S, R, H, q, scale, out, None, ws, n, None)

    need = B.tf_paged_mla_shared_workspace_bytes(None, 3, 2, 16, [1000, 2048, 30], [2, 1], [640, 0])
    assert need > 0
    for bad in ({"pool": None}, {"G": 0}, {"G": 4, "g": (1, 1, 1, 0), "f": (0, 0, 0, 0)}, {"g": (2, 2)}, {"g": (3, 0)},
                {"g": (4, -1)}, {"g": (2, 0)}, {"S": 0}, {"H": 0}, {"mp": 0}, {"q": BASE + 8}, {"out": None},
                {"scale": 0.0}, {"ws": None}, {"ws": BASE + 64}):
        assert call(**bad) == B.TF_E_ARG, bad
    for bad in ({"cache": -1}, {"lens": (1000, 2049, 30)}, {"lens": (1000, 2048, 1)}, {"f": (1000, 0)}, {"f": (-1, 0)},
                {"f": (640, 30)}, {"pt": None, "mp": 11}):
        assert call(**bad) == B.TF_E_RANGE, bad
    assert call(n=need - 1) == B.TF_E_NOMEM
    # 512 streams and a group that shares: one entry too many
    S = 512
    assert call(S=S, lens=(640,) * S, g=(2,) + (1,) * (S - 2), G=S - 1, f=(64,) + (0,) * (S - 2), mp=4) == B.TF_E_UNSUPPORTED
    assert B.tf_paged_mla_shared_workspace_bytes(None, S, 2, 16, [640] * S, [2] + [1] * (S - 2), [64] + [0] * (S - 2)) == 0
    assert B.tf_paged_mla_shared_workspace_bytes(None, S - 1, 2, 16, [640] * (S - 1), [S - 1], [64]) > 0


def test_workspace_sizes(L):
    slot = 64 * 512 * 4
    # blocks: one row with eight tiles or fewer than a range's worth is one CTA's
    assert B.tf_paged_mla_blocks_workspace_bytes(None, 1, 1, 16, [64], 8) == 0
    # at most two partial slots a CTA
    n = B.tf_paged_mla_blocks_workspace_bytes(None, 1, 2048, 64, [102048], 32)
    assert 0 < n <= 2 * 240 * (slot + 64 * 8) + 256
    # shared: nothing shared and one short stream needs none; a group always merges
    assert B.tf_paged_mla_shared_workspace_bytes(None, 1, 1, 16, [64], [1], [0]) == 0
    assert B.tf_paged_mla_shared_workspace_bytes(None, 2, 1, 16, [64, 64], [2], [64]) > 0
    for bad in ({"R": 0}, {"H": 200}):
        kw = {"R": 1, "H": 16} | bad
        assert B.tf_paged_mla_blocks_workspace_bytes(None, 1, kw["R"], kw["H"], [64], 8) == 0
        assert B.tf_paged_mla_shared_workspace_bytes(None, 1, kw["R"], kw["H"], [64], [1], [0]) == 0
    assert B.tf_paged_mla_blocks_workspace_bytes(None, 1, 1, 16, [64], 0) == 0
    assert B.tf_paged_mla_shared_workspace_bytes(None, 1, 1, 16, [64], [1], [65]) == 0


class _FakePool:
    def __init__(self):
        self.handle, self.num_pages = _pool(4, 1), 4


def test_binding_refuses_what_the_library_cannot_see(L):
    p = _FakePool()
    bf = dict(dtype=torch.bfloat16)
    bk, q = torch.zeros(4, 8, 576, **bf), torch.zeros(2, 1, 16, 576, **bf)
    out, lse = torch.zeros(2, 1, 16, 512, **bf), torch.zeros(2, 1, 16)
    pt, blk = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 1, 4, dtype=torch.int32)
    bad = [
        lambda: B.tf_block_keys_update(p, 0, pt, 2, [0], [64, 64], bk),
        lambda: B.tf_block_keys_update(p, 0, pt, 2, [0, 0], [64, 64], bk.float()),
        lambda: B.tf_block_keys_update(p, 0, pt, 2, [0, 0], [64, 64], bk[:3]),
        lambda: B.tf_block_scores(p, bk, pt, 2, [64, 64, 64], q, 0.1, torch.zeros(2, 4)),
        lambda: B.tf_block_scores(p, bk, pt, 2, [64, 64], q, 0.1, torch.zeros(1, 4)),
        lambda: B.tf_block_scores(p, bk, pt, 2, [64, 640], q, 0.1, torch.zeros(2, 16)[:, :8]),
        lambda: B.tf_block_scores(p, bk, pt, 2, [64, 64], q, 0.1, torch.zeros(2, 4), w=torch.zeros(2, 15)),
        lambda: B.tf_block_scores(p, bk, pt, 2, [64, 64], q, 0.1, torch.zeros(2, 4), nblk=torch.zeros(2)),
        lambda: B.tf_paged_mla_attend_blocks(p, 0, pt, 2, [64, 64], blk.long(), q, 0.1, out, lse),
        lambda: B.tf_paged_mla_attend_blocks(p, 0, pt, 2, [64, 64], blk[:1], q, 0.1, out, lse),
        lambda: B.tf_paged_mla_attend_blocks(p, 0, pt, 2, [64], blk, q, 0.1, out, lse),
        lambda: B.tf_paged_mla_attend_blocks(p, 0, pt, 2, [64, 64], blk, q.half(), 0.1, out, lse),
        lambda: B.tf_paged_mla_attend_blocks(p, 0, pt, 2, [64, 64], blk, q, 0.1, out[:, :, :8], lse),
        lambda: B.tf_paged_mla_attend_shared(p, 0, pt, 2, [64, 64], [2], [0, 0], q, 0.1, out, lse),
        lambda: B.tf_paged_mla_attend_shared(p, 0, pt, 2, [64], [2], [0], q, 0.1, out, lse),
        lambda: B.tf_paged_mla_attend_shared(p, 0, pt, 2, [64, 64], [2], [0], q, 0.1, out, lse[0]),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(B.TFError) as e:
            f()
        assert e.value.code == B.TF_E_ARG, i


@pytest.mark.parametrize("pt", [torch.zeros(2, 2, dtype=torch.int64), torch.zeros(1, 2, dtype=torch.int32),
                                torch.zeros(3, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)[:, :2]],
                         ids=["int64", "one_row", "short", "strided"])
def test_binding_refuses_a_table_of_another_form(L, pt):
    p = _FakePool()
    bf = dict(dtype=torch.bfloat16)
    bk, q = torch.zeros(4, 8, 576, **bf), torch.zeros(2, 1, 16, 576, **bf)
    out, blk = torch.zeros(2, 1, 16, 512, **bf), torch.zeros(2, 1, 4, dtype=torch.int32)
    for f in (lambda: B.tf_block_keys_update(p, 0, pt, 2, [0, 0], [64, 64], bk),
              lambda: B.tf_block_scores(p, bk, pt, 2, [64, 64], q, 0.1, torch.zeros(2, 4)),
              lambda: B.tf_paged_mla_attend_blocks(p, 0, pt, 2, [64, 64], blk, q, 0.1, out),
              lambda: B.tf_paged_mla_attend_shared(p, 0, pt, 2, [64, 64], [2], [0], q, 0.1, out)):
        with pytest.raises(B.TFError) as e:
            f()
        assert e.value.code == B.TF_E_ARG


def test_binding_refuses_no_streams(L):
    p = _FakePool()
    bf = dict(dtype=torch.bfloat16)
    with pytest.raises(B.TFError) as e:
        B.tf_block_scores(p, torch.zeros(4, 8, 576, **bf), None, 2, [], torch.zeros(0, 1, 16, 576, **bf), 0.1,
                          torch.zeros(0, 4))
    assert e.value.code == B.TF_E_ARG


def test_header_is_strict_c99(L, tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "tf_blocks.h"\nint main(void) { return TF_BLOCK_ROWS - 64; }\n')
    cc = shutil.which("gcc") or "gcc"
    r = subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), "-c",
                        str(src), "-o", str(tmp_path / "t.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
