"""Attention of packed prompts: what a causal row does not see, NaN and infinities included, does not reach it.

The expectation follows from the definition: a row that does not see a key keeps its output and lse, whatever key and
value are; a row that sees it has, in the value's column, what the sum of positive weights times the values gives (NaN for
a NaN or infinities of both signs, else the infinity; a weight below fp32's range times an infinity is NaN, which the
tests' scores do not come near).  Bits stay but for one case: where a row does not see a value, but the last row of its
query tile (128 rows: tokens times the heads of a key head) sees one of its 128-key tile or of a later one, the value's
column may be rounded in another way.
Both results are then within (u + 2^-10) sum p|v| + u |ref| of the definition (u = 2^-8; test_gpu_prompt.py has the reasons;
2^-10 is far above the scores' and sums' errors of these inputs), so within 4.5 u sum p|v| of each other.
"""
import numpy as np
import pytest
import torch

from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from tests.gpu_common import bits
from tests.test_gpu_prompt import call, make

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
WIDTHS = [(192, 128, True), (192, 128, False), (128, 128, False), (64, 64, False)]
SHAPES = [  # nq, nk, H, Hkv
    ([128], [192], 1, 1),             # query tiles and key tiles do not line up
    ([200], [300], 2, 2),
    ([130], [131], 2, 1),
    ([300], [301], 6, 2),             # three heads to a key head: 42 tokens a query tile
    ([700], [700], 3, 1),
    ([70], [333], 16, 2),             # eight
    ([9], [200], 64, 1),              # two tokens a query tile, one a block's last
    ([5], [129], 128, 1),             # one token a query tile
    ([400], [250], 2, 2),             # rows that see no key at all
    ([300], [90], 6, 2),
    ([300], [6000], 2, 2),            # keys split
    ([2], [40001], 64, 1),
    ([3, 260, 1, 40], [140, 400, 77, 40], 4, 2),
]


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()
    B.lib()


@pytest.fixture(scope="module")
def pool():
    return B.KVPool(1, 1)


def places(n, m):
    """Keys of a stream of n rows and m keys where something can go wrong: the last ones, tiles' borders, the middle."""
    at = {m - 1, m - 2, m - n // 2, m - n + 1, m // 128 * 128, m // 128 * 128 - 1, m - 17, 0}
    return sorted({j for j in at if 0 <= j < m})


def sees(nq, nk, s, key):
    """Rows of the packed call that see key `key` of stream s."""
    off = sum(nq[:s])
    rows = torch.zeros(sum(nq), dtype=torch.bool)
    for i in range(nq[s]):
        rows[off + i] = key < nk[s] - nq[s] + i + 1
    return rows


def share_a_tile(nq, nk, s, key, G):
    """Rows of the packed call whose query tile is multiplied with the key's tile."""
    off, per = sum(nq[:s]), 128 // G
    rows = torch.zeros(sum(nq), dtype=torch.bool)
    for i in range(nq[s]):
        last = min(nq[s], (i // per + 1) * per) - 1
        rows[off + i] = key < -(-max(0, nk[s] - nq[s] + last + 1) // 128) * 128
    return rows


def close(got, clean, size):
    """Outputs that are rounded in another way; `size`: those of |v|, about sum p|v|."""
    return ((got.float() - clean.float()).abs() <= 4.5 * 2.0 ** -8 * size.float()).all()


def expected(pairs):
    """The sum of positive weights times (value or None): NaN, an infinity, or None where all are finite."""
    v = [x for x in pairs if x is not None]
    if not v:
        return None
    return NAN if any(x != x for x in v) or {INF, -INF} <= set(v) else v[0]


@pytest.mark.parametrize("dqk,dv,kr", WIDTHS)
@pytest.mark.parametrize("nq,nk,H,Hkv", SHAPES)
def test_a_value_reaches_the_rows_that_see_it(pool, nq, nk, H, Hkv, dqk, dv, kr):
    q, k, v, rot = make(nq, nk, H, Hkv, dqk, dv, kr, seed=31)
    clean, lclean = call(pool, nq, nk, q, k, v, kr=rot)
    size, _ = call(pool, nq, nk, q, k, v.abs(), kr=rot)
    G, h = H // Hkv, Hkv - 1
    s = len(nq) // 2 if len(nq) > 1 else 0
    base = sum(nk[:s])
    for n, key in enumerate(places(nq[s], nk[s])):
        y = v.clone()
        kinds = {3: NAN, 20: INF, dv - 1: -INF}
        for c, x in kinds.items():
            y[base + key, h, c] = x
        out, lse = call(pool, nq, nk, q, k, y, kr=rot)
        assert torch.equal(lse, lclean)                       # (NaN compares unequal: there is none)
        seen = sees(nq, nk, s, key)
        changed = torch.tensor(bits(out) != bits(clean))
        near = share_a_tile(nq, nk, s, key, G) & ~seen
        assert not changed[~seen & ~near].any(), key
        assert close(out[near], clean[near], size[near]), key
        assert not changed[:, :h * G].any()
        for c in range(dv):
            if c not in kinds:
                assert not changed[:, :, c].any(), (key, c)
        got = out[seen][:, h * G:].cpu()
        for c, x in kinds.items():
            assert torch.isnan(got[..., c]).all() if x != x else (got[..., c] == x).all(), (key, c)


@pytest.mark.parametrize("dqk,dv,kr", WIDTHS)
@pytest.mark.parametrize("nq,nk,H,Hkv", SHAPES)
def test_several_values_at_once(pool, nq, nk, H, Hkv, dqk, dv, kr):
    """Every later half of a column's values not finite, and infinities of both signs met one after another."""
    q, k, v, rot = make(nq, nk, H, Hkv, dqk, dv, kr, seed=32)
    clean, lclean = call(pool, nq, nk, q, k, v, kr=rot)
    size = call(pool, nq, nk, q, k, v.abs(), kr=rot)[0].float().cpu()
    G = H // Hkv
    y = v.clone()
    marks = {}                                                # (stream, column) -> [(key, value)]
    for s in range(len(nq)):
        base, n, m = sum(nk[:s]), nq[s], nk[s]
        first = max(0, m - n // 2 - 1)
        for c, keys in {1: [(j, NAN) for j in range(first, m)], 2: [(max(0, m - n // 3 - 1), INF), (m - 1, -INF)], dv - 2: [(m - 1, INF), (max(0, m - 2), INF)]}.items():
            for j, x in keys:
                y[base + j, 0, c] = x
            marks[s, c] = dict(keys).items()
    out, lse = call(pool, nq, nk, q, k, y, kr=rot)
    assert torch.equal(lse, lclean)
    got, ref = out[:, :G].float().cpu(), clean[:, :G].float().cpu()
    for (s, c), keys in marks.items():
        off = sum(nq[:s])
        for i in range(nq[s]):
            e = expected([x for j, x in keys if j < nk[s] - nq[s] + i + 1])
            g = got[off + i, :, c]
            assert close(g, ref[off + i, :, c], size[off + i, :G, c]) if e is None else torch.isnan(g).all() if e != e else (g == e).all(), (s, i, c, e)
    other = [c for c in range(dv) if c not in (1, 2, dv - 2)]
    assert np.array_equal(bits(out[..., other]), bits(clean[..., other])) and np.array_equal(bits(out[:, G:]), bits(clean[:, G:]))


@pytest.mark.parametrize("dqk,dv,kr", WIDTHS)
@pytest.mark.parametrize("nq,nk,H,Hkv", SHAPES)
def test_a_key_reaches_the_rows_that_see_it(pool, nq, nk, H, Hkv, dqk, dv, kr):
    q, k, v, rot = make(nq, nk, H, Hkv, dqk, dv, kr, seed=33)
    clean, lclean = call(pool, nq, nk, q, k, v, kr=rot)
    s = len(nq) - 1
    for key in places(nq[s], nk[s])[-3:]:
        seen = sees(nq, nk, s, key)
        for x in (NAN, INF, -INF):
            y = k.clone()
            y[sum(nk[:s]) + key, :, 0] = x
            out, lse = call(pool, nq, nk, q, y, v, kr=rot)
            assert np.array_equal(bits(out[~seen]), bits(clean[~seen])) and torch.equal(lse[~seen], lclean[~seen])
            if x != x:
                assert torch.isnan(out[seen]).all() and torch.isnan(lse[seen]).all()


def test_many_items_and_long_ones(pool):
    """More items than SMs, whose blocks follow one another on an SM: bad values in some streams and heads only."""
    nq = [513, 1, 300, 40, 2048, 129, 64, 257]
    nk = [513, 900, 333, 40, 2100, 129, 650, 258]
    H = 40
    q, k, v, rot = make(nq, nk, H, H, 192, 128, True, seed=34)
    clean, lclean = call(pool, nq, nk, q, k, v, kr=rot)
    size, _ = call(pool, nq, nk, q, k, v.abs(), kr=rot)
    y = v.clone()
    bad = [(0, 0, 511), (2, 7, 200), (4, 39, 2099), (4, 3, 300), (4, 3, 1500), (5, 20, 128), (7, 11, 129)]
    first = {}
    for s, h, key in bad:
        y[sum(nk[:s]) + key, h, 77] = NAN
        first[s, h] = min(key, first.get((s, h), 1 << 30))
    want = torch.zeros(sum(nq), H, dtype=torch.bool)
    for (s, h), key in first.items():
        want[:, h] |= sees(nq, nk, s, key)
    for _ in range(3):
        out, lse = call(pool, nq, nk, q, k, y, kr=rot)
        assert torch.equal(lse, lclean)
        assert torch.equal(torch.isnan(out[..., 77]).cpu(), want)
        changed = torch.tensor(bits(out) != bits(clean))
        assert not changed[..., :77].any() and not changed[..., 78:].any()
        near = torch.zeros_like(want)
        for s, h, key in bad:
            near[:, h] |= share_a_tile(nq, nk, s, key, 1)
        assert not changed[..., 77][~near].any()
        assert close(out[..., 77].cpu()[~want], clean[..., 77].cpu()[~want], size[..., 77].cpu()[~want])


def test_values_without_a_mask(pool):
    """Not causal: every row sees every value."""
    nq, nk, H = [70, 3], [200, 5], 2
    q, k, v, _ = make(nq, nk, H, H, 128, 128, seed=35)
    clean, _ = call(pool, nq, nk, q, k, v, causal=False)
    y = v.clone()
    y[199, 1, 5], y[3, 1, 6] = NAN, INF
    out, _ = call(pool, nq, nk, q, k, y, causal=False)
    changed = torch.tensor(bits(out) != bits(clean))
    assert changed[:70, 1, 5:7].all() and changed.sum() == 140
    assert torch.isnan(out[:70, 1, 5]).all() and (out[:70, 1, 6] == INF).all()


def test_a_row_made_again_over_many_keys(pool):
    """Rows that are made again over 131,072 keys take longer than the kernel's other waits are allowed to: those know."""
    n = m = 131072
    H = 8
    assert B.tf_prompt_plan_info([n], [m], H, H, 192, 128, sms=152)["splits"] == 1
    q, k, v, rot = make([n], [m], H, H, 192, 128, True, seed=36)
    clean, lclean = call(pool, [n], [m], q, k, v, kr=rot)
    size = call(pool, [128], [m], q[-128:], k, v.abs(), kr=rot)[0]
    v[m - 1, 3, 64] = NAN
    out, lse = call(pool, [n], [m], q, k, v, kr=rot)
    assert torch.equal(lse, lclean)
    nan = torch.isnan(out)
    assert nan.sum() == 1 and nan[n - 1, 3, 64]
    changed = out.view(torch.int16) != clean.view(torch.int16)
    assert not changed[:-128].any() and not changed[:, :3].any() and not changed[:, 4:].any()
    assert not changed[..., :64].any() and not changed[..., 65:].any()
    assert close(out[-128:-1, 3, 64], clean[-128:-1, 3, 64], size[:-1, 3, 64])
