"""GPU parity of block keys, block scores and attention over listed blocks, and of attention of streams that
share a prefix, against fp64 definitions, through the C-ABI.

Tolerances count roundings.  u = 2^-8 is half a bf16 step (relative), f = 2^-23 an fp32 sum's step (the tensor
cores may cut where others round).  A score s = scale q.k of n products is off by at most e = scale n f sum|q k|.
A softmax weight is then off by the factor exp(2 e), its bf16 form by u more, and the output by u once more:
|out - ref| <= (u + 2 e + 2^-18) sum_j p_j |c_j| + u |ref|, the 2^-18 for the exponentials and the sums of the
partials.  lse is off by at most e + 2^-18 max(1, |lse|).
"""
import numpy as np
import pytest
import torch

from oracle import blocks as K
from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from paged_mla_kv_gb300 import synth as Y
from paged_mla_kv_gb300.harness import Resident, bf16_tensor
from tests.gpu_common import bits, no_device_error

pytestmark = pytest.mark.gpu

U, F = 2.0 ** -8, 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()
    B.lib()


def values(b):
    return Y.bf16_bits_to_f32(b).astype(np.float64)


def rows64(w, s, fp8=False):
    """Stream s's rows as the pool holds them, float64."""
    lat, rope = w.stream_rows(0, s)
    if fp8:
        from oracle import fp8 as F8
        x = F8.dequantize_rows(*F8.quantize_rows(Y.bf16_bits_to_f32(lat)))
        lat = values(Y.f32_to_bf16_bits(np.asarray(x, np.float32)))
    else:
        lat = values(lat)
    return lat, values(rope)


def check_row(got, lse, q, lat, rope, rows, scale):
    """One query row's heads: got [H][512], lse [H] against attention over `rows` in fp64."""
    ref, lref = K.attend_rows(q, lat, rope, rows, scale)
    if len(rows) == 0:
        assert not got.any() and np.all(np.isneginf(lse))
        return
    k = np.concatenate([lat[rows], rope[rows]], 1)
    s = scale * (q @ k.T)
    e = (scale * 577 * F * (np.abs(q) @ np.abs(k).T)).max(1)
    p = np.exp(s - lref[:, None])
    tol = (U + 2 * e[:, None] + 2.0 ** -18) * (p @ np.abs(k[:, :512])) + U * np.abs(ref)
    assert np.all(np.abs(got - ref) <= tol), float((np.abs(got - ref) / tol).max())
    assert np.all(np.abs(lse - lref) <= e + 2.0 ** -18 * np.maximum(1, np.abs(lref)))


def host(t):
    return t.double().cpu().numpy()


# ---- block keys --------------------------------------------------------------------------------

def key_tol(ref, rows):
    # 64 fp32 additions, a division, one rounding to bf16
    return U * np.abs(ref) + 66 * F * np.abs(rows).mean(0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("windowed", [False, True])
def test_block_keys(fp8, windowed):
    lens = [1, 63, 64, 65, 511, 512, 513, 1301]
    w = Y.custom("keys", 81 + fp8, lens=lens, R=1, H=16)
    res = Resident(w, windowed=windowed, fp8=fp8)
    bk = torch.full((res.pool.num_pages, 8, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    B.tf_block_keys_update(res.pool, 0, res.pt, res.max_pages, [0] * 8, lens, bk)
    got = host(bk)
    no_device_error(res.pool)
    seen = np.zeros(got.shape[:2], bool)
    for s, n in enumerate(lens):
        lat, rope = rows64(w, s, fp8)
        ref = K.block_keys(lat, rope)
        for b in range(len(ref)):
            pg = int(res.pt_host[s, b // 8])
            seen[pg, b % 8] = True
            r = np.concatenate([lat, rope], 1)[64 * b:64 * b + 64]
            assert np.all(np.abs(got[pg, b % 8] - ref[b]) <= key_tol(ref[b], r)), (s, b)
    assert np.all(got[~seen] == 7.0)     # other blocks are left as they were


@pytest.mark.parametrize("fp8", [False, True])
def test_block_keys_of_new_rows_only(fp8):
    lens, start = [700, 1301, 64, 900], [699, 1100, 64, 0]
    w = Y.custom("keysn", 85, lens=lens, R=1, H=16)
    res = Resident(w, fp8=fp8)
    full = torch.zeros((res.pool.num_pages, 8, 576), dtype=torch.bfloat16, device="cuda")
    B.tf_block_keys_update(res.pool, 0, res.pt, res.max_pages, [0] * 4, lens, full)
    part = torch.full_like(full, 7.0)
    B.tf_block_keys_update(res.pool, 0, res.pt, res.max_pages, start, lens, part)
    a, b = host(full), host(part)
    for s, n in enumerate(lens):
        for k in range(K.blocks_of(n)):
            pg = int(res.pt_host[s, k // 8])
            fresh = start[s] < n and k >= start[s] // 64
            assert np.array_equal(b[pg, k % 8], a[pg, k % 8]) if fresh else np.all(b[pg, k % 8] == 7.0), (s, k)
    # a shorter length averages only the rows below it
    B.tf_block_keys_update(res.pool, 0, res.pt, res.max_pages, [640, 0, 0, 0], [650, 0, 0, 0], part)
    lat, rope = rows64(w, 0, fp8)
    r = np.concatenate([lat, rope], 1)[640:650]
    assert np.all(np.abs(host(part)[int(res.pt_host[0, 1]), 2] - r.mean(0)) <= key_tol(r.mean(0), r))


def test_block_keys_bad_page_is_recorded():
    w = Y.custom("keysb", 86, lens=[600, 600], R=1, H=16)
    res = Resident(w)
    bk = torch.full((res.pool.num_pages, 8, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    pt = res.pt.clone()
    pt[0, 1] = res.pool.num_pages
    B.tf_block_keys_update(res.pool, 0, pt, res.max_pages, [0, 0], [600, 600], bk)
    assert res.pool.last_error() == (B.TF_E_DEVICE, res.pool.num_pages)
    got = host(bk)
    assert np.all(got[int(res.pt_host[0, 1])] == 7.0) and not np.any(got[int(res.pt_host[1, 1]), :2] == 7.0)


# ---- block scores ------------------------------------------------------------------------------

def run_scores(res, w, bk, q, weights=None, sink=1, local=1, extra=0, lens=None):
    lens = w.lens if lens is None else lens
    cols = K.blocks_of(int(max(lens)))
    ld = -(-cols // 4) * 4 + 4 * extra
    R = q.shape[1]
    x = torch.full((len(lens) * R, ld), 7.0, device="cuda")
    n = torch.full((len(lens) * R,), -5, dtype=torch.int32, device="cuda")
    B.tf_block_scores(res.pool, bk, res.pt, res.max_pages, lens, q, w.scale, x, w=weights, nblk=n, sink=sink, local=local)
    no_device_error(res.pool)
    return x, n, cols


@pytest.mark.parametrize("lens,R,H,sink,local,weighted", [
    ([1], 1, 1, 0, 1, False), ([64], 1, 16, 1, 1, True), ([65, 1, 9000], 1, 64, 0, 1, False),
    ([8192, 8193, 300], 2, 16, 1, 2, True), ([20000, 513], 2, 128, 2, 3, True), ([5000], 7, 100, 0, 1, False),
    ([3000, 2000], 33, 5, 1, 1, True), ([9000, 300], 131, 64, 1, 4, True), ([700], 700, 20, 3, 1, False),
    ([17000] * 3, 3, 96, 0, 5, True), ([700], 7, 85, 0, 1, True), ([9000], 60, 5, 0, 1, False), ([600], 9, 127, 1, 1, True),
    ([40000], 500, 8, 1, 1, True)])
def test_block_scores(lens, R, H, sink, local, weighted):
    w = Y.custom("sc", 90 + R + H, lens=lens, R=R, H=H)
    res = Resident(w, caches=[])
    g = torch.Generator(device="cuda").manual_seed(R * 1000 + H)
    bk = torch.randn((res.pool.num_pages, 8, 576), generator=g, device="cuda").bfloat16()
    q = torch.randn((w.S, R, H, 576), generator=g, device="cuda").bfloat16()
    wt = torch.randn((w.S, R, H), generator=g, device="cuda") if weighted else None
    x, n, cols = run_scores(res, w, bk, q, wt, sink, local, extra=2)
    xs, keys, qs = host(x), host(bk), host(q)
    assert np.all(xs[:, cols:] == 7.0)
    for s, L in enumerate(lens):
        nb = K.blocks_of(L)
        k = np.stack([keys[int(res.pt_host[s, b // 8]), b % 8] for b in range(nb)])
        ws = None if wt is None else host(wt)[s]
        ref = K.block_scores(qs[s], k, L, ws, w.scale, sink, local)
        got = xs[s * R:(s + 1) * R]
        assert np.all(np.isneginf(got[:, nb:cols]))
        assert n[s * R:(s + 1) * R].tolist() == [(L - R + r) // 64 + 1 for r in range(R)]
        fin = np.isfinite(ref)
        assert np.array_equal(got[:, :nb][~fin], ref[~fin])
        # 576 products and H terms, each rounded; the scale once more
        mag = np.abs(qs[s]) @ np.abs(k).T
        mag = (mag if ws is None else mag * np.abs(ws)[..., None]).sum(1)
        assert np.all(np.abs(got[:, :nb][fin] - ref[fin]) <= (w.scale * (580 + H) * F * mag)[fin])


def test_block_scores_same_bits_and_null_outputs():
    w = Y.custom("scn", 97, lens=[5000, 70], R=2, H=16)
    res = Resident(w, caches=[], windowed=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    bk = torch.randn((res.pool.num_pages, 8, 576), generator=g, device="cuda").bfloat16()
    q = torch.randn((2, 2, 16, 576), generator=g, device="cuda").bfloat16()
    a, _, cols = run_scores(res, w, bk, q)
    x = torch.zeros_like(a)
    B.tf_block_scores(res.pool, bk, None, res.max_pages, w.lens, q, w.scale, x)
    assert torch.equal(a[:, :cols], x[:, :cols])
    ones = torch.ones((2, 2, 16), device="cuda")
    B.tf_block_scores(res.pool, bk, None, res.max_pages, w.lens, q, w.scale, x, w=ones)
    assert torch.equal(a[:, :cols], x[:, :cols])


def test_block_scores_bad_page_leaves_the_rest():
    w = Y.custom("scb", 98, lens=[5000], R=1, H=16)
    res = Resident(w, caches=[])
    bk = torch.randn((res.pool.num_pages, 8, 576), device="cuda").bfloat16()
    q = torch.randn((1, 1, 16, 576), device="cuda").bfloat16()
    a, _, cols = run_scores(res, w, bk, q)
    pt = res.pt.clone()
    pt[0, 3] = -1
    x = torch.zeros_like(a)
    B.tf_block_scores(res.pool, bk, pt, res.max_pages, w.lens, q, w.scale, x)
    assert res.pool.last_error() == (B.TF_E_DEVICE, -1)
    keep = [b for b in range(cols) if b // 8 != 3]
    assert torch.equal(a[:, keep], x[:, keep])


# ---- attention over listed blocks --------------------------------------------------------------

def run_blocks(res, w, blk, q=None, scale=None, stream=None):
    S, R, H = w.S, w.R, w.H
    q = res.q() if q is None else q
    out = torch.full((S, R, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((S, R, H), 7.0, device="cuda")
    n = B.tf_paged_mla_blocks_workspace_bytes(res.pool, S, R, H, res.lens, blk.shape[-1])
    ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda") if n else None   # NaN wherever it is read unwritten
    B.tf_paged_mla_attend_blocks(res.pool, 0, res.pt, res.max_pages, res.lens, blk, q, w.scale if scale is None else scale,
                                 out, lse, ws, stream=stream)
    return out, lse


def check_blocks(res, w, blk, out, lse, fp8=False, rows=None, scale=None):
    o, l, b, q = host(out), host(lse), blk.view(w.S, w.R, -1).cpu().numpy(), values(w.q(0))
    for s in range(w.S):
        lat, rope = rows64(w, s, fp8)
        for r in range(w.R) if rows is None else rows:
            pos = int(w.lens[s]) - w.R + r
            lst = b[s, r][:min(b.shape[-1], pos // 64 + 1)].tolist()
            check_row(o[s, r], l[s, r], q[s, r], lat, rope, K.rows_of_list(lst, pos), w.scale if scale is None else scale)


def random_lists(w, k, seed, holes=True):
    g = np.random.default_rng(seed)
    blk = np.full((w.S, w.R, k), -1, np.int32)
    for s in range(w.S):
        for r in range(w.R):
            own = (int(w.lens[s]) - w.R + r) // 64
            m = min(k, own + 1)
            lst = g.permutation(own + 1)[:m]
            if holes and m > 2:
                lst[g.integers(0, m)] = -1
            blk[s, r, :m] = lst
    return torch.from_numpy(blk).cuda()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,R,H,k", [
    ([1], 1, 1, 1), ([64, 65, 2], 1, 16, 4), ([513, 3000, 127, 64], 2, 64, 5), ([5000, 700], 1, 128, 17),
    ([4000, 600], 2, 96, 64), ([2000, 1000], 40, 20, 9), ([1500], 300, 64, 12), ([700] * 9, 3, 5, 3), ([20000] * 2, 1, 64, 300)])
def test_attend_blocks(lens, R, H, k, fp8):
    w = Y.custom("bl", 110 + H + k, lens=lens, R=R, H=H, q_std=1.0, value_std=0.5)
    res = Resident(w, fp8=fp8)            # rows behind a stream's last hold NaN
    blk = random_lists(w, k, H + k)
    out, lse = run_blocks(res, w, blk)
    no_device_error(res.pool)
    check_blocks(res, w, blk, out, lse, fp8, rows=None if R <= 40 else [0, 1, 63, 64, 150, 298, 299])
    again = run_blocks(res, w, blk)
    assert np.array_equal(bits(out), bits(again[0])) and torch.equal(lse, again[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_attend_blocks_lists_that_leave_nothing_repeat_or_look_ahead(fp8):
    w = Y.custom("ble", 120, lens=[1000, 1000, 1000, 1000, 300], R=70, H=16, q_std=1.0, value_std=0.5)
    res = Resident(w, fp8=fp8)
    blk = torch.full((5, 70, 6), -1, dtype=torch.int32, device="cuda")   # stream 0: no block at all
    blk[1] = 3                                                            # the same block six times
    blk[2] = torch.tensor([15, 14, -1, 15, 13, 14], dtype=torch.int32)    # some rows' blocks lie behind them
    blk[3, ::2, 0] = 15                                                   # alone: rows before 960 see nothing
    blk[4] = torch.tensor([4, 3, 2, 1, 0, -1], dtype=torch.int32)         # the last block holds 44 rows
    out, lse = run_blocks(res, w, blk)
    no_device_error(res.pool)
    check_blocks(res, w, blk, out, lse, fp8)
    assert torch.isneginf(lse[0]).all() and not out[0].any()


def test_attend_blocks_empty_rows_that_are_cut():
    """Rows without a key in units that several CTAs share: zero and -inf come out of the merge too."""
    w = Y.custom("blc", 121, lens=[30000] * 3, R=1, H=16)
    res = Resident(w)
    blk = torch.full((3, 1, 400), -1, dtype=torch.int32, device="cuda")
    blk[1, 0, 399] = 5
    out, lse = run_blocks(res, w, blk)
    no_device_error(res.pool)
    check_blocks(res, w, blk, out, lse)
    assert torch.isneginf(lse[0]).all() and not out[0].any() and torch.isfinite(lse[1]).all()


@pytest.mark.parametrize("windowed", [False, True])
def test_attend_blocks_of_every_block_is_the_dense_call(windowed):
    w = Y.custom("bld", 122, lens=[3000, 130, 777], R=2, H=64, q_std=1.0, value_std=0.5)
    res = Resident(w, windowed=windowed)
    nb = K.blocks_of(3000)
    blk = torch.arange(nb, dtype=torch.int32, device="cuda").expand(3, 2, nb).contiguous()
    for s, L in enumerate(w.lens):
        blk[s, :, K.blocks_of(int(L)):] = -1
    out, lse = run_blocks(res, w, blk)
    o2, l2 = res.attend(res.q())
    check_blocks(res, w, blk, out, lse)
    check_dense(w, o2, l2)


def test_attend_blocks_infinite_and_large_scores():
    """Scores hundreds apart: the running maximum moves, weights that vanish stay zero."""
    w = Y.custom("blx", 123, lens=[2000], R=1, H=16, q_std=8.0, value_std=2.0)
    res = Resident(w)
    blk = random_lists(w, 20, 3, holes=False)
    out, lse = run_blocks(res, w, blk, scale=0.5)
    no_device_error(res.pool)
    o, l, q = host(out), host(lse), values(w.q(0))
    lat, rope = rows64(w, 0)
    rows = K.rows_of_list(blk[0, 0].tolist(), 1999)
    # e is large here: the weights' tolerance is exp(2 e) - 1 of the two best rows' gap
    ref, lref = K.attend_rows(q[0, 0], lat, rope, rows, 0.5)
    k = np.concatenate([lat, rope], 1)[rows]
    e = (0.5 * 577 * F * (np.abs(q[0, 0]) @ np.abs(k).T)).max(1)
    p = np.exp(0.5 * (q[0, 0] @ k.T) - lref[:, None])
    tol = (U + np.expm1(2 * e)[:, None] + 2.0 ** -18) * (p @ np.abs(k[:, :512])) + U * np.abs(ref)
    assert np.all(np.abs(o[0, 0] - ref) <= tol) and np.all(np.abs(l[0, 0] - lref) <= e + 2.0 ** -18 * np.abs(lref))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", ["below", "behind", "page"])
def test_attend_blocks_bad_entries_are_recorded(bad, fp8):
    w = Y.custom("blb", 124, lens=[1000, 1000], R=1, H=16)
    res = Resident(w, fp8=fp8)
    blk = random_lists(w, 8, 5, holes=False)
    good = run_blocks(res, w, blk)
    no_device_error(res.pool)
    kept = blk.clone()
    pt = res.pt
    if bad == "below":
        blk[0, 0, 3] = -2
        want = -2
    elif bad == "behind":
        blk[0, 0, 3] = 16        # the stream's blocks are 0 .. 15
        want = 16
    else:
        res.pt = pt.clone()
        res.pt[0, :] = res.pool.num_pages + 3
        want = res.pool.num_pages + 3
    run_blocks(res, w, blk)
    assert res.pool.last_error() == (B.TF_E_DEVICE, want)
    res.pt = pt
    again = run_blocks(res, w, kept)     # the context goes on
    no_device_error(res.pool)
    assert np.array_equal(bits(good[0]), bits(again[0]))


# ---- the four calls of a step, and graphs ------------------------------------------------------

class Step:
    """append, block keys, scores, top-k, attention over the chosen blocks: one decode step."""

    def __init__(self, w, k, fp8=False):
        self.w, self.k = w, k
        self.res = res = Resident(w, fp8=fp8, caches=[0])
        self.bk = torch.zeros((res.pool.num_pages, 8, 576), dtype=torch.bfloat16, device="cuda")
        B.tf_block_keys_update(res.pool, 0, res.pt, res.max_pages, [0] * w.S, w.lens, self.bk)
        self.cols = K.blocks_of(int(w.lens.max()))
        rows = w.S * w.R
        self.scores = torch.zeros((rows, -(-self.cols // 4) * 4), device="cuda")
        self.nblk = torch.zeros((rows,), dtype=torch.int32, device="cuda")
        self.idx = torch.zeros((rows, k), dtype=torch.int32, device="cuda")
        self.val = torch.zeros((rows, k), device="cuda")
        self.q = res.q()
        self.out = torch.zeros((w.S, w.R, w.H, 512), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.zeros((w.S, w.R, w.H), device="cuda")
        n = B.tf_paged_mla_blocks_workspace_bytes(res.pool, w.S, w.R, w.H, w.lens, k)
        self.ws = torch.zeros((max(n, 256),), dtype=torch.uint8, device="cuda")
        n = B.tf_topk_workspace_bytes(rows, self.cols, k)
        self.wk = torch.zeros((max(n, 256),), dtype=torch.uint8, device="cuda")
        self.new = res.current_rows(0)

    def run(self, stream=None):
        w, res = self.w, self.res
        B.tf_paged_append(res.pool, 0, res.pt, res.max_pages, w.lens - w.R, *self.new, stream=stream)
        B.tf_block_keys_update(res.pool, 0, res.pt, res.max_pages, w.lens - w.R, w.lens, self.bk, stream=stream)
        B.tf_block_scores(res.pool, self.bk, res.pt, res.max_pages, w.lens, self.q, w.scale, self.scores, nblk=self.nblk,
                          sink=1, local=2, stream=stream)
        B.tf_topk_blocked(self.scores, self.k, self.idx, self.val, lens=self.nblk, n=self.cols, ws=self.wk, stream=stream)
        B.tf_paged_mla_attend_blocks(res.pool, 0, res.pt, res.max_pages, w.lens, self.idx, self.q, w.scale, self.out,
                                     self.lse, self.ws, stream=stream)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_step_of_block_sparse_attention(fp8):
    w = Y.custom("step", 130, lens=[5000, 1234, 200, 64], R=2, H=16, q_std=1.0, value_std=0.5)
    st = Step(w, 6, fp8)
    st.run()
    no_device_error(st.res.pool)
    idx, val = st.idx.cpu().numpy(), st.val.cpu().numpy()
    for s in range(w.S):
        for r in range(w.R):
            own = (int(w.lens[s]) - w.R + r) // 64
            got = [b for b in idx[s * w.R + r].tolist() if b >= 0]
            assert len(set(got)) == len(got) == min(6, own + 1)
            assert {0, own, max(0, own - 1)} <= set(got)
            # the rest are the best of the scores
            x = st.scores[s * w.R + r, :own + 1].cpu().numpy()
            assert set(got) == set(sorted(range(own + 1), key=lambda b: (-x[b], b))[:6])
    check_blocks(st.res, w, st.idx, st.out, st.lse, fp8)


def test_a_step_in_a_graph_on_a_side_stream_replays_the_eager_bits():
    w = Y.custom("stepg", 131, lens=[5000, 700, 9000], R=1, H=64)
    st = Step(w, 16)
    st.run()
    torch.cuda.synchronize()
    eager = [t.clone() for t in (st.bk, st.scores, st.idx, st.out, st.lse)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        st.run(stream=torch.cuda.current_stream().cuda_stream)
    for _ in range(3):
        for t in (st.scores, st.idx, st.out, st.lse, st.ws):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (st.bk, st.scores, st.idx, st.out, st.lse)):
            assert torch.equal(a, b)
    no_device_error(st.res.pool)


def test_two_calls_on_two_streams_at_once():
    w = Y.custom("two", 132, lens=[4000, 900], R=2, H=64)
    a, b = Step(w, 8), Step(w, 8)
    a.run()
    b.q = (b.q.float() * 2).bfloat16()
    b.run()
    torch.cuda.synchronize()
    want = [x.out.clone() for x in (a, b)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        a.run(stream=s1.cuda_stream)
        b.run(stream=s2.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


# ---- streams that share a prefix ---------------------------------------------------------------

class Prefixed(Y.Workload):
    """Streams whose prefix ends inside a page: the page is each one's own, its first rows are the same."""

    def page_rows(self, cache, s, page):
        lat, rope = super().page_rows(cache, s, page)
        first, p = self.extra["prefix"][s]
        n = p - page * 512
        if s != first and 0 < n < 512:
            l0, r0 = super().page_rows(cache, first, page)
            lat[:n], rope[:n] = l0[:n], r0[:n]
        return lat, rope


def shared_workload(name, seed, groups, R, H):
    """groups: (prefix rows, [own rows...]); pages under a prefix are held by reference."""
    extra = []
    lens, share, sizes, prefixes, first = [], [], [], [], 0
    for p, own in groups:
        for i, n in enumerate(own):
            lens.append(p + n)
            share.append((first, p // 512) if i else (0, 0))
            extra.append((first, p))
        sizes.append(len(own))
        prefixes.append(p)
        first += len(own)
    w = Y.custom(name, seed, lens=lens, R=R, H=H, share=share, q_std=1.0, value_std=0.5)
    w.__class__ = Prefixed
    w.extra["prefix"] = extra
    return w, sizes, prefixes


def run_shared(res, w, sizes, prefixes):
    q = res.q()
    out = torch.full((w.S, w.R, w.H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((w.S, w.R, w.H), 7.0, device="cuda")
    n = B.tf_paged_mla_shared_workspace_bytes(res.pool, w.S, w.R, w.H, w.lens, sizes, prefixes)
    ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda") if n else None
    B.tf_paged_mla_attend_shared(res.pool, 0, res.pt, res.max_pages, w.lens, sizes, prefixes, q, w.scale, out, lse, ws)
    return out, lse


def check_dense(w, out, lse, fp8=False, rows=None):
    o, l, q = host(out), host(lse), values(w.q(0))
    for s in range(w.S):
        lat, rope = rows64(w, s, fp8)
        for r in range(w.R) if rows is None else rows:
            check_row(o[s, r], l[s, r], q[s, r], lat, rope, np.arange(int(w.lens[s]) - w.R + r + 1), w.scale)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("groups,R,H", [
    ([(512, [1, 2, 3, 700])], 1, 16),                 # 64 columns of four streams
    ([(1024, [5] * 9)], 1, 20),                       # column groups that cut streams
    ([(512, [1, 64, 65]), (0, [300]), (2048, [2, 600])], 2, 64),
    ([(1536, [3, 3])], 3, 128), ([(512, [40, 90, 41])], 40, 5), ([(2560, [1] * 30)], 1, 5),
    ([(512, [100]), (1024, [100])], 1, 64),           # groups of one stream share nothing
    ([(16384, [1, 900, 17])], 1, 64),
    ([(1000, [300, 90]), (0, [100, 70])], 70, 64),      # chunks of rows behind a prefix that ends inside a page
    ([(520, [1, 2, 3])], 1, 64), ([(960, [33] * 5), (64, [700])], 4, 16),
    ([(4096, [9, 70, 600]), (2560, [5, 5])], 5, 128)])   # rows that many columns read: FP8 pages are expanded first
def test_attend_shared(groups, R, H, fp8):
    w, sizes, prefixes = shared_workload("sh", 140 + R + H, groups, R, H)
    res = Resident(w, fp8=fp8)
    out, lse = run_shared(res, w, sizes, prefixes)
    no_device_error(res.pool)
    check_dense(w, out, lse, fp8)
    again = run_shared(res, w, sizes, prefixes)
    assert np.array_equal(bits(out), bits(again[0])) and torch.equal(lse, again[1])


@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 65, 512, 575, 576, 1000, 1024])
def test_attend_shared_prefix_of_any_length(prefix):
    """Streams that share 1,024 rows, told to use fewer of them; at 1,024 the first has no row of its own."""
    w, _, _ = shared_workload("shp", 150, [(1024, [0, 1, 70])], 1, 16)
    res = Resident(w)
    out, lse = run_shared(res, w, [3], [prefix])
    no_device_error(res.pool)
    check_dense(w, out, lse)


def test_attend_shared_windows():
    """A null table: the shared rows are the same bytes in each stream's own window."""
    w, sizes, prefixes = shared_workload("shw", 151, [(1024, [30, 200, 513])], 1, 16)
    res = Resident(w, windowed=True)
    out, lse = run_shared(res, w, sizes, prefixes)
    no_device_error(res.pool)
    check_dense(w, out, lse)


def test_attend_shared_reads_the_prefix_through_the_first_table():
    w, sizes, prefixes = shared_workload("sht", 152, [(1024, [30, 200, 513])], 1, 16)
    res = Resident(w)
    good = run_shared(res, w, sizes, prefixes)
    kept = res.pt
    res.pt = kept.clone()
    res.pt[1:, :2] = -1                      # the others' entries of shared pages are not looked at
    out, lse = run_shared(res, w, sizes, prefixes)
    no_device_error(res.pool)
    assert np.array_equal(bits(out), bits(good[0])) and torch.equal(lse, good[1])
    res.pt[0, 1] = -7
    run_shared(res, w, sizes, prefixes)
    assert res.pool.last_error() == (B.TF_E_DEVICE, -7)
    res.pt = kept
    again = run_shared(res, w, sizes, prefixes)
    no_device_error(res.pool)
    assert np.array_equal(bits(again[0]), bits(good[0]))


def test_attend_shared_many_streams():
    """The largest batch the entries allow: 340 streams in pairs, and 511 that share one prompt."""
    w, sizes, prefixes = shared_workload("shm", 153, [(512, [1 + i % 5, 70]) for i in range(170)], 1, 2)
    res = Resident(w)
    out, lse = run_shared(res, w, sizes, prefixes)
    no_device_error(res.pool)
    check_dense(w, out, lse)
    w, sizes, prefixes = shared_workload("shn", 154, [(512, [1 + i % 3 for i in range(511)])], 1, 1)
    res = Resident(w)
    out, lse = run_shared(res, w, sizes, prefixes)
    no_device_error(res.pool)
    check_dense(w, out, lse)


def test_attend_shared_in_a_graph():
    w, sizes, prefixes = shared_workload("shg", 155, [(8192, [5, 100, 300, 64])], 2, 64)
    res = Resident(w)
    q = res.q()
    out = torch.zeros((w.S, w.R, w.H, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((w.S, w.R, w.H), device="cuda")
    n = B.tf_paged_mla_shared_workspace_bytes(res.pool, w.S, w.R, w.H, w.lens, sizes, prefixes)
    ws = torch.zeros((n,), dtype=torch.uint8, device="cuda")

    def run():
        B.tf_paged_mla_attend_shared(res.pool, 0, res.pt, res.max_pages, w.lens, sizes, prefixes, q, w.scale, out, lse, ws)

    run()
    torch.cuda.synchronize()
    want = out.clone(), lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(2):
        out.zero_(), lse.zero_(), ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ---- pools ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True])
def test_calls_on_a_batch_invariant_pool(fp8):
    """The plans are the calls' own whatever the pool's flags."""
    w, sizes, prefixes = shared_workload("inv", 160, [(1024, [30, 200, 513])], 2, 64)
    out = []
    for invariant in (False, True):
        res = Resident(w, fp8=fp8, invariant=invariant)
        a = run_shared(res, w, sizes, prefixes)
        b = run_blocks(res, w, random_lists(w, 9, 4))
        no_device_error(res.pool)
        out.append([bits(a[0]), bits(b[0]), a[1].cpu().numpy(), b[1].cpu().numpy()])
    for x, y in zip(*out):
        assert np.array_equal(x, y)


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_past_four_gigabytes(fp8):
    """A stream whose pages lie anywhere in a pool of 9 GB: the bits of a small pool."""
    w = Y.custom("far", 161, lens=[1500, 700], R=2, H=16, q_std=1.0, value_std=0.5)
    got = []
    for pages in (8, 9_400_000_000 // (B.PAGE_BYTES_FP8 if fp8 else B.PAGE_BYTES_BF16)):
        res = Resident.__new__(Resident)
        res.w, res.windowed, res.device, res.max_pages = w, False, "cuda", w.max_pages
        res.pool = B.KVPool(1, pages, seed=5, fp8=fp8)
        ids = np.concatenate([res.pool.take(3), res.pool.take(2)])
        if pages > 8:      # both ends and what is between
            ids = np.array([pages - 1, 1, pages - 2, pages // 2, pages - 3], np.int32)
        pt = np.full((2, 3), -1, np.int32)
        pt[0], pt[1, :2] = ids[:3], ids[3:]
        res.pt, res.pt_host, res.lens = torch.from_numpy(pt).cuda(), pt, np.asarray(w.lens, np.int64)
        for s in range(2):
            res.append_rows(0, s, 0, int(w.lens[s]))
        bk = torch.zeros((pages, 8, 576), dtype=torch.bfloat16, device="cuda")
        B.tf_block_keys_update(res.pool, 0, res.pt, 3, [0, 0], w.lens, bk)
        x, n, cols = run_scores(res, w, bk, res.q())
        out, lse = run_blocks(res, w, random_lists(w, 6, 2))
        sh = run_shared(res, w, [1, 1], [512, 0])
        no_device_error(res.pool)
        keys = torch.stack([bk[int(pt[s, b // 8]), b % 8] for s in range(2) for b in range(K.blocks_of(int(w.lens[s])))])
        got.append([bits(keys), x[:, :cols].cpu().numpy(), bits(out), lse.cpu().numpy(), bits(sh[0])])
        del res, bk
    for a, b in zip(*got):
        assert np.array_equal(a, b)
