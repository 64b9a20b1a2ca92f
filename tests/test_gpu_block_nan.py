"""NaN and infinities through block scores and attention over listed blocks: a value that is not a number
stays one, in the columns that it belongs to and nowhere else.  Tolerances as in test_gpu_blocks."""
import numpy as np
import pytest
import torch

from oracle import blocks as K
from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from paged_mla_kv_gb300 import synth as Y
from paged_mla_kv_gb300.harness import Resident
from tests.gpu_common import no_device_error
from tests.test_gpu_blocks import check_row, host, random_lists, rows64, run_blocks, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()
    B.lib()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("S,H,n,k", [
    (1, 16, 2048, 8),       # a unit on a cluster of several CTAs
    (64, 64, 1500, 32),     # on two, each merging half of the columns
    (3, 96, 1500, 8),       # two head groups a row
    (1, 16, 20000, 300),    # cut, merged by a combine pass
    (300, 16, 600, 2)])     # whole units
def test_nan_queries_give_nan(S, H, n, k, fp8):
    w = Y.custom("nanq", 170 + k, lens=[n] * S, R=1, H=H, q_std=1.0, value_std=0.5)
    res = Resident(w, fp8=fp8)
    q = res.q()
    q[0, 0, 3, 5] = float("nan")
    q[S - 1, 0, H - 1, 570] = float("nan")
    blk = random_lists(w, k, k, holes=False)
    out, lse = run_blocks(res, w, blk, q=q)
    no_device_error(res.pool)
    bad = torch.zeros((S, 1, H), dtype=torch.bool)
    bad[0, 0, 3] = bad[S - 1, 0, H - 1] = True
    assert torch.equal(torch.isnan(lse).cpu(), bad)
    assert torch.isnan(out.cpu()[bad]).all() and torch.isfinite(out.cpu()[~bad].float()).all()
    o, l, b, qs = host(out), host(lse), blk.cpu().numpy(), values(w.q(0))
    for s in {0, S - 1}:
        lat, rope = rows64(w, s, fp8)
        fine = ~bad[s, 0].numpy()
        check_row(o[s, 0][fine], l[s, 0][fine], qs[s, 0][fine], lat, rope, K.rows_of_list(b[s, 0].tolist(), n - 1), w.scale)


@pytest.mark.parametrize("H,weighted", [(64, False), (64, True), (8, True), (20, False), (20, True), (5, True), (1, False)])
def test_scores_of_nan_and_infinite_keys(H, weighted):
    """A block whose key was never averaged must not pass for an ordinary one."""
    lens, R = [5000, 700], 3
    w = Y.custom("nans", 175, lens=lens, R=R, H=H)
    res = Resident(w, caches=[])
    g = torch.Generator(device="cuda").manual_seed(H)
    bk = torch.randn((res.pool.num_pages, 8, 576), generator=g, device="cuda").bfloat16()
    q = torch.randn((2, R, H, 576), generator=g, device="cuda").bfloat16()
    wt = torch.randn((2, R, H), generator=g, device="cuda") if weighted else None
    nan, inf = float("nan"), float("inf")

    def key(s, b):
        return bk[int(res.pt_host[s, b // 8]), b % 8]

    key(0, 5)[:] = nan                      # every product
    key(0, 9)[575] = nan
    key(1, 2)[0] = nan
    key(0, 20)[7], key(0, 21)[7] = inf, -inf
    key(0, 22)[3], key(0, 22)[4] = inf, inf   # inf - inf for some heads
    q[0, 1, 0, 100] = nan                   # one head of one row: all its scores
    if weighted:
        wt[0, 2, H - 1] = inf
    cols = K.blocks_of(5000)
    x = torch.zeros((2 * R, -(-cols // 4) * 4), device="cuda")
    B.tf_block_scores(res.pool, bk, res.pt, res.max_pages, lens, q, w.scale, x, w=wt, sink=1, local=2)
    no_device_error(res.pool)
    xs, keys, qs = host(x), host(bk), host(q)
    with np.errstate(invalid="ignore"):
        for s, n in enumerate(lens):
            nb = K.blocks_of(n)
            k = np.stack([keys[int(res.pt_host[s, b // 8]), b % 8] for b in range(nb)])
            ws = None if wt is None else host(wt)[s]
            ref = K.block_scores(qs[s], k, n, ws, w.scale, 1, 2)
            got = xs[s * R:(s + 1) * R, :nb]
            assert np.array_equal(np.isnan(got), np.isnan(ref))
            fin = np.isfinite(ref)
            odd = ~fin & ~np.isnan(ref)
            assert np.array_equal(got[odd], ref[odd])
            mag = np.abs(qs[s]) @ np.abs(k).T
            mag = (mag if ws is None else mag * np.abs(ws)[..., None]).sum(1)
            assert np.all(np.abs(got[fin] - ref[fin]) <= (w.scale * (580 + H) * 2.0 ** -23 * mag)[fin])
    assert np.isnan(xs[0, 5]) and np.isnan(xs[2, 9]) and np.isnan(xs[3, 2]) and np.isnan(xs[1, 1:70]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,R,H,k", [(200, 4, 16, 4), (1000, 3, 64, 16), (1500, 130, 16, 8), (20000, 2, 64, 300), (1300, 70, 64, 21)])
def test_rows_behind_a_query_may_be_nan(n, R, H, k, fp8):
    """A query attends the rows up to its own.  What the rows behind it hold, in its own block or in listed ones that
    begin behind it, does not reach its output."""
    w = Y.custom("behind", 176 + R, lens=[n, n - 3], R=R, H=H, q_std=1.0, value_std=0.5)
    res = Resident(w, fp8=fp8)
    g = np.random.default_rng(R)
    blk = random_lists(w, k, k, holes=False)
    own = torch.tensor([[(int(L) - R + r) // 64 for r in range(R)] for L in w.lens], dtype=torch.int32, device="cuda")
    last = torch.tensor([[(int(L) - 1) // 64] for L in w.lens], dtype=torch.int32, device="cuda")
    seen = torch.clamp_max(own + 1, k)                        # the entries that are read
    place = torch.from_numpy(g.permutation(k)).cuda()
    pick = place[None, None].expand(2, R, k) < seen[..., None]
    first = torch.where(pick, place[None, None].expand(2, R, k), k).amin(-1, keepdim=True).long()
    blk.scatter_(2, first, own[..., None])                    # each row lists its own block
    if k > 2:
        blk[..., 0] = torch.where((own != last) & (first[..., 0] != 0), last.expand(2, R), blk[..., 0])   # and some the last one
    good = run_blocks(res, w, blk)
    no_device_error(res.pool)
    bad = R // 2                                              # the rows behind query row `bad` - 1 are NaN
    for s in range(2):
        lat = torch.full((1, R - bad, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
        rope = torch.full((1, R - bad, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        B.tf_paged_append(res.pool, 0, res.stream_pt(s), res.max_pages, [int(w.lens[s]) - R + bad], lat, rope)
    out, lse = run_blocks(res, w, blk)
    no_device_error(res.pool)
    assert torch.equal(out[:, :bad], good[0][:, :bad]) and torch.equal(lse[:, :bad], good[1][:, :bad])
    assert torch.isnan(out[:, bad:]).any(-1).all()            # the others see their own row
