"""Work plans of listed blocks and shared prefixes (host arithmetic, no GPU): what they cost, and that they deal
out every tile of every unit once."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()


# The largest batches that the calls take: a plan holds runs of equal units, so it takes neither their memory
# nor their time.
@pytest.mark.parametrize("call", [
    "B.tf_paged_mla_blocks_workspace_bytes(None, 1, 1 << 30, 1, [1 << 30], 1)",
    "B.tf_paged_mla_blocks_workspace_bytes(None, 1, 1 << 30, 1, [(1 << 31) - 1], 4096)",
    "B.tf_paged_mla_blocks_workspace_bytes(None, 512, 1 << 14, 128, [1 << 20] * 512, 100)",
    "B.tf_paged_mla_shared_workspace_bytes(None, 2, 1 << 22, 128, [1 << 30] * 2, [2], [1 << 20])"])
def test_the_largest_plans_are_small(call):
    code = ("import resource, time\nfrom paged_mla_kv_gb300 import binding as B\n"
            "B.tf_paged_mla_blocks_workspace_bytes(None, 1, 1, 16, [64], 8)\n"
            "a, t = resource.getrusage(resource.RUSAGE_SELF).ru_maxrss, time.perf_counter()\n"
            f"n = {call}\n"
            "t = time.perf_counter() - t\nprint(n, resource.getrusage(resource.RUSAGE_SELF).ru_maxrss - a, t)")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-500:]
    n, kib, seconds = r.stdout.split()
    assert int(n) >= 0 and int(kib) < 8192 and float(seconds) < 0.25, r.stdout


SEG = 3      # what a segment weighs in tiles
MERGING = 7  # and a combine pass at most


def check_plan(p, nt, sms):
    """nt: the tiles of each unit.  The bounds deal them out in order, within the SMs and evenly."""
    b = [(int(x) >> 32, int(x) & 0xffffffff) for x in p["bounds"]]
    assert p["units"] == len(nt) and len(b) == p["ctas"] + 1 and 1 <= p["ctas"] <= sms
    assert b[0] == (0, 0) and b[-1] == (len(nt), 0)
    assert all(t < nt[u] for u, t in b[:-1] if t)
    assert p["cut"] == int(any(t for _, t in b))
    at = np.concatenate([[0], np.cumsum(nt)])
    tiles = np.diff([at[u] + t for u, t in b])
    if p["merge"]:
        k = p["merge"]
        assert 2 <= k <= 8 and p["ctas"] == k * len(nt) and len(nt) <= sms // k
        for v, n in enumerate(nt):      # a unit's CTAs are neighbours; short units may leave some without a tile
            assert b[v * k] == (v, 0) and tiles[v * k:v * k + k].sum() == n
            assert tiles[v * k:v * k + k].max() <= -(-n // k)
        assert p["slots"] >= p["ctas"]
        return
    assert np.all(tiles > 0)
    if p["cut"]:
        assert p["slots"] >= 2 * p["ctas"] or p["slots"] >= len(nt) + p["ctas"]
    segs = np.array([b[i + 1][0] - b[i][0] + (1 if b[i + 1][1] else 0) for i in range(p["ctas"])])
    n = max(1, min(sms, -(-sum(nt) // 2)))
    assert (tiles + SEG * segs).max() <= (sum(nt) + SEG * len(nt)) / n + 1 + SEG + MERGING


def spread(g, lo, hi):
    return int(np.exp(g.uniform(np.log(lo), np.log(hi + 0.99))))


@pytest.mark.parametrize("seed", range(4))
def test_listed_block_plans(seed):
    g = np.random.default_rng(seed)
    merged = cut = 0
    for _ in range(100):
        S, R, H = spread(g, 1, 80), spread(g, 1, 40 if g.random() < 0.7 else 500), int(g.choice([1, 16, 64, 65, 96, 128]))
        lens = np.maximum(R, g.integers(1, spread(g, 64, 60000) + 1, S)).tolist()
        k, sms = spread(g, 1, 300), int(g.choice([152, 152, 240, 7, 1]))
        p = B.tf_paged_mla_blocks_plan_info(S, R, H, lens, k, sms)
        nt = [min(k, (n - R + r) // 64 + 1) for n in lens for r in range(R) for _ in range(-(-H // 64))]
        check_plan(p, nt, sms)
        merged += p["merge"] > 0
        cut += p["cut"] and not p["merge"]
    assert merged > 5 and cut > 5


@pytest.mark.parametrize("seed", range(4))
def test_shared_prefix_plans(seed):
    g = np.random.default_rng(100 + seed)
    for _ in range(100):
        G, R, H = spread(g, 1, 12), spread(g, 1, 30), int(g.choice([1, 5, 16, 64, 96, 128]))
        sizes = g.integers(1, 12, G).tolist()
        prefixes = [spread(g, 1, 20000) if g.random() < 0.8 else 0 for _ in range(G)]
        lens = [f + R - 1 + int(g.integers(0, 900)) if f else R + int(g.integers(0, 900)) for f, n in zip(prefixes, sizes) for _ in range(n)]
        sms = int(g.choice([152, 240, 7]))
        p = B.tf_paged_mla_shared_plan_info(len(lens), R, H, lens, sizes, prefixes, sms)
        own, shared, s = [], [], 0
        split = R * H % 64 != 0
        for f, n in zip(prefixes, sizes):
            whole = f // 64 if n > 1 and split else 0
            if whole:
                shared += [whole] * -(-n * R * H // 64)
            for _ in range(n):
                own += [-(-lens[s] // 64) - whole] * -(-R * H // 64)
                s += 1
        check_plan(p, [t for t in own + shared if t], sms)
        assert not p["merge"]


def test_of_equal_loads_the_one_with_fewer_partials():
    """24 streams behind 4,096 shared rows: 19 tiles a CTA on 144 CTAs or on 152."""
    lens = [4104 + 100 * (s * 618 % 1000) // 1000 for s in range(24)]
    assert B.tf_paged_mla_shared_plan_info(24, 1, 64, lens, [24], [4096], 152)["ctas"] == 144


def test_plans_size_the_workspace():
    for S, R, H, n, k in ((64, 1, 64, 32768, 32), (1, 2048, 64, 102048, 32), (1, 1, 16, 2048, 8), (3, 2, 96, 5000, 20), (1, 1, 16, 64, 8)):
        slots = B.tf_paged_mla_blocks_plan_info(S, R, H, [n] * S, k)["slots"]
        need = B.tf_paged_mla_blocks_workspace_bytes(None, S, R, H, [n] * S, k)
        assert need == slots * (64 * 512 * 4) + -(-slots * 64 * 8 // 256) * 256
    slots = B.tf_paged_mla_shared_plan_info(8, 1, 16, [9000] * 8, [8], [8192])["slots"]
    assert B.tf_paged_mla_shared_workspace_bytes(None, 8, 1, 16, [9000] * 8, [8], [8192]) == slots * (64 * 512 * 4 + 64 * 8)


def test_plan_queries_refuse():
    L, n = B.lib(), np.asarray([640, 640], np.int64)
    g, f, info = np.asarray([2], np.int32), np.asarray([64], np.int64), B.tf_unit_plan()
    pn, pg, pf, pi = n.ctypes.data, g.ctypes.data, f.ctypes.data, ctypes.byref(info)

    def blocks(S=2, R=1, H=16, lens=pn, k=4, info=pi):
        return L.tf_paged_mla_blocks_plan_info(S, R, H, lens, k, 152, info, None)

    def shared(S=2, R=1, H=16, lens=pn, g=pg, G=1, f=pf, info=pi):
        return L.tf_paged_mla_shared_plan_info(S, R, H, lens, g, G, f, 152, info, None)

    assert blocks() == B.TF_OK and info.units == 2 and shared() == B.TF_OK and info.units == 3
    for bad in ({"S": 0}, {"R": 0}, {"H": 129}, {"lens": None}, {"info": None}):
        assert blocks(**bad) == B.TF_E_ARG and shared(**bad) == B.TF_E_ARG, bad
    assert blocks(k=0) == B.TF_E_ARG and shared(G=2) == B.TF_E_ARG and shared(g=None) == B.TF_E_ARG
    assert blocks(R=641) == B.TF_E_RANGE and shared(R=641) == B.TF_E_RANGE
    assert blocks(R=1 << 24, H=128) == B.TF_E_UNSUPPORTED
    many = np.full(512, 640, np.int64)
    gs, fs = np.asarray([2] + [1] * 510, np.int32), np.asarray([64] + [0] * 510, np.int64)
    assert shared(S=512, lens=many.ctypes.data, g=gs.ctypes.data, G=511, f=fs.ctypes.data) == B.TF_E_UNSUPPORTED
