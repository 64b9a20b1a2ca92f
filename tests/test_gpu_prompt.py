"""GPU parity of the attention of packed prompts against the fp64 definition, through the C-ABI.

Tolerances count roundings, as in test_gpu_blocks.py.  u = 2^-8 is half a bf16 step (relative), f = 2^-23 an fp32
sum's step (the tensor cores may cut where others round).  A score s = scale q.k of n products is off by at most
scale n f sum|q k|; its exponent, taken from s c - m c, by 2^-22 max|s| more; together e.  A softmax weight is then
off by the factor exp(2 e), its bf16 form by u more, and the output by u once more:
|out - ref| <= (u + 2 e + 2^-18) sum_j p_j |v_j| + u |ref|, the 2^-18 for the exponentials and the sums of the
partials.  lse is off by at most e + 2^-18 max(1, |lse|).
"""
import numpy as np
import pytest
import torch

from oracle import prompt as O
from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from tests.gpu_common import bits, no_device_error

pytestmark = pytest.mark.gpu

U, F = 2.0 ** -8, 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()
    B.lib()


@pytest.fixture(scope="module")
def pool():
    return B.KVPool(1, 1)


def host(t):
    return t.double().cpu().numpy()


def make(nq, nk, H, Hkv, dqk, dv, kr=False, seed=0, sharp=1.0):
    """Inputs of a call; with kr the keys and values are slices of one joint projection."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    K = sum(nk)
    q = (torch.randn((sum(nq), H, dqk), generator=g, device="cuda") * sharp).bfloat16()
    if not kr:
        return q, rnd(K, Hkv, dqk), rnd(K, Hkv, dv), None
    kv = rnd(K, Hkv, dqk - 64 + dv)
    return q, kv[..., :dqk - 64], kv[..., dqk - 64:], rnd(K, 64)


def call(pool, nq, nk, q, k, v, kr=None, causal=True, scale=None, out=None, lse=None, stream=None):
    H, Hkv, dqk, dv = q.shape[1], v.shape[1], q.shape[2], v.shape[2]
    out = torch.full((q.shape[0], H, dv), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    lse = torch.full((q.shape[0], H), float("nan"), device="cuda") if lse is None else lse
    n = B.tf_prompt_workspace_bytes(nq, nk, H, Hkv, dqk, dv, causal)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    B.tf_prompt_attend(pool, nq, nk, q, k, v, dqk ** -0.5 if scale is None else scale, out, lse=lse, kr=kr, causal=causal, ws=ws,
                       stream=stream)
    no_device_error(pool)
    return out, lse


def full_keys(k, kr):
    k = host(k)
    return k if kr is None else np.concatenate([k, np.broadcast_to(host(kr)[:, None], k.shape[:2] + (64,))], -1)


def check(nq, nk, q, k, v, kr, causal, out, lse, scale=None, streams=None, rows=None):
    """Streams' outputs against the definition, all rows or `rows` of them (from the end)."""
    scale = q.shape[2] ** -0.5 if scale is None else scale
    G = q.shape[1] // v.shape[1]
    a = b = 0
    for s, (n, m) in enumerate(zip(nq, nk)):
        if n and (streams is None or s in streams):
            r0 = 0 if rows is None else max(0, n - rows)
            kk, vv = full_keys(k[b:b + m], None if kr is None else kr[b:b + m]), host(v[b:b + m])
            qq = host(q[a + r0:a + n])
            ref, lref = O.attend(qq, kk, vv, scale, causal)
            got, gl = host(out[a + r0:a + n]), host(lse[a + r0:a + n])
            for h in range(q.shape[1]):
                x = kk[:, h // G]
                sc = scale * (qq[:, h] @ x.T)
                if causal:
                    sc = np.where(np.arange(m)[None] <= np.arange(m - (n - r0), m)[:, None], sc, -np.inf)
                some = np.isfinite(lref[:, h])
                assert not got[~some, h].any() and np.all(np.isneginf(gl[~some, h])), (s, h)
                if not some.any():
                    continue
                e = (scale * (q.shape[2] + 1) * F * (np.abs(qq[:, h]) @ np.abs(x).T)).max(1)
                e = e + 2.0 ** -22 * np.abs(np.where(np.isfinite(sc), sc, 0)).max(1)
                p = np.exp(sc[some] - lref[some, h][:, None])
                e = e[some]
                tol = (U + 2 * e[:, None] + 2.0 ** -18) * (p @ np.abs(vv[:, h // G])) + U * np.abs(ref[some, h])
                err = np.abs(got[some, h] - ref[some, h])
                assert np.all(err <= tol), (s, h, float((err / tol).max()))
                assert np.all(np.abs(gl[some, h] - lref[some, h]) <= e + 2.0 ** -18 * np.maximum(1, np.abs(lref[some, h]))), (s, h)
        a, b = a + n, b + m


@pytest.mark.parametrize("dqk,dv,kr", [(192, 128, True), (192, 128, False), (128, 128, False), (128, 128, True), (64, 64, False)])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 256, 257, 400])
def test_one_prompt(pool, n, dqk, dv, kr):
    x = make([n], [n], 2, 2, dqk, dv, kr, seed=n)
    out, lse = call(pool, [n], [n], *x)
    check([n], [n], *x, True, out, lse)


@pytest.mark.parametrize("dqk,dv", [(192, 128), (128, 128), (64, 64)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("row", [130, 255, 511, 699])
def test_own_values_that_are_not_finite(pool, dqk, dv, value, row):
    """A key leaves the rows before it as they are; so do values, but for rows whose last key lies in their tile."""
    n = 700
    q, k, v, _ = make([n], [n], 3, 3, dqk, dv, seed=1)
    clean, lclean = call(pool, [n], [n], q, k, v)
    for x, first in ((k, row), (v, row // 128 * 128)):
        y = x.clone()
        y[row, 1] = value
        out, lse = call(pool, [n], [n], q, *((y, v) if x is k else (k, y)))
        same = (bits(out) == bits(clean)).all(-1) & (lse.cpu() == lclean.cpu()).numpy()
        assert same[:, [0, 2]].all() and same[:first, 1].all(), first
        if value != value:
            assert torch.isnan(out[row:, 1]).all()


def test_groups_of_heads(pool):
    """Keys and values of all heads that do not fit L2 side by side: seven heads in groups of three, three and one."""
    nq, nk, H = [300, 3], [60000, 70], 7
    x = make(nq, nk, H, H, 64, 64, seed=70)
    out, lse = call(pool, nq, nk, *x)
    check(nq, nk, *x, True, out, lse)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (2, 1), (3, 1), (10, 2), (8, 1), (16, 2), (64, 1), (128, 1), (48, 1), (100, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_grouped_heads(pool, H, Hkv, causal):
    nq, nk = [37, 1, 5], [300, 1, 5]
    x = make(nq, nk, H, Hkv, 128, 128, seed=H)
    out, lse = call(pool, nq, nk, *x, causal=causal)
    check(nq, nk, *x, causal, out, lse)


@pytest.mark.parametrize("dqk,dv,kr", [(192, 128, True), (128, 128, False), (64, 64, False)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk", [
    ([5, 0, 300, 1, 129], [5, 9, 300, 1, 129]),          # a stream without rows
    ([7, 3, 130], [0, 3, 0]),                            # streams without keys
    ([0, 0], [5, 0]), ([4], [0]),                        # no rows at all; no keys at all
    ([300, 140, 9], [77, 1, 3]),                         # more queries than keys: rows that see none
    ([1, 2, 1, 3], [1000, 129, 4097, 513]),              # decode and drafts
    ([33, 260], [1111, 2000]),                           # chunks behind prefixes
])
def test_packed(pool, nq, nk, causal, dqk, dv, kr):
    x = make(nq, nk, 4, 2, dqk, dv, kr, seed=3)
    out, lse = call(pool, nq, nk, *x, causal=causal)
    check(nq, nk, *x, causal, out, lse)


def test_many_streams(pool):
    r = np.random.default_rng(5)
    nq = [int(x) for x in r.integers(0, 40, 512)]
    nk = [n + int(x) for n, x in zip(nq, r.integers(0, 60, 512))]
    x = make(nq, nk, 2, 1, 64, 64, seed=6)
    out, lse = call(pool, nq, nk, *x)
    check(nq, nk, *x, True, out, lse)


@pytest.mark.parametrize("nq,nk,H,Hkv", [([1], [20000], 8, 1), ([1, 1], [9000, 700], 16, 2), ([300], [6000], 2, 2), ([2], [40001], 64, 1),
                                         ([1, 260, 3], [5000, 260, 12345], 4, 4)])
@pytest.mark.parametrize("dqk,dv,kr", [(192, 128, True), (128, 128, False), (64, 64, False)])
def test_split_keys(pool, nq, nk, H, Hkv, dqk, dv, kr):
    info = B.tf_prompt_plan_info(nq, nk, H, Hkv, dqk, dv)
    assert info["splits"] > 1 and info["slots"] > 0
    x = make(nq, nk, H, Hkv, dqk, dv, kr, seed=8)
    out, lse = call(pool, nq, nk, *x)
    check(nq, nk, *x, True, out, lse, rows=4)


@pytest.mark.parametrize("sharp", [0.0, 8.0, 60.0])
@pytest.mark.parametrize("nk", [300, 3000])
def test_sharp_scores(pool, sharp, nk):
    """Equal scores, and maxima that move by far more than the rescaling's step."""
    nq = [200]
    q, k, v, _ = make(nq, [nk], 2, 1, 128, 128, seed=9, sharp=sharp)
    k = (k.float() * torch.linspace(0.1, 2.0, nk, device="cuda")[:, None, None]).bfloat16()   # later keys dominate
    out, lse = call(pool, nq, [nk], q, k, v)
    check(nq, [nk], q, k, v, None, True, out, lse)


def test_what_others_hold_does_not_count(pool):
    """NaN and infinities in other streams' rows, behind the tensors and in rows of no stream's output."""
    nq, nk = [5, 40, 130], [77, 40, 333]
    for H, Hkv, dqk, dv, kr in [(4, 2, 192, 128, True), (10, 2, 128, 128, False), (2, 2, 64, 64, False)]:
        clean = make(nq, nk, H, Hkv, dqk, dv, kr, seed=11)
        ref, lref = call(pool, nq, nk, *clean)
        q, k, v, kk = [None if t is None else torch.full((t.shape[0] + 300,) + tuple(t.shape[1:]), float("nan"), dtype=t.dtype, device="cuda")
                       for t in clean]
        for big, t in zip((q, k, v, kk), clean):
            if t is not None:
                big[:t.shape[0]] = t
        bad = [q[:sum(nq)], k[:sum(nk)], v[:sum(nk)], None if kk is None else kk[:sum(nk)]]
        bad[0][5:45] = float("nan")              # the second stream
        bad[1][77:117], bad[2][77:117] = float("inf"), float("nan")
        if kk is not None:
            bad[3][77:117] = float("nan")
        out, lse = call(pool, nq, nk, *bad)
        for a, b in ((0, 5), (45, 175)):
            assert np.array_equal(bits(out[a:b]), bits(ref[a:b])) and torch.equal(lse[a:b], lref[a:b])
        assert torch.isnan(out[5:45]).all()


def test_strided_heads_and_outputs(pool):
    nq, nk, H, Hkv, d = [70, 9], [200, 9], 6, 3, 128
    q, k, v, _ = make(nq, nk, H, Hkv, d, d, seed=12)
    ref, lref = call(pool, nq, nk, q, k, v)
    qkv = torch.zeros((209, H + 2 * Hkv, d + 8), dtype=torch.bfloat16, device="cuda")
    qs = qkv[:79, :H, :d]
    qs.copy_(q)
    ks, vs = qkv[:, H:H + Hkv, 8:], qkv[:, H + Hkv:, :d]
    ks.copy_(k)
    vs.copy_(v)
    kt = k.transpose(0, 1).contiguous().transpose(0, 1)       # head by head
    big = torch.full((79, H + 1, d + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    for kk in (ks, kt):
        out, lse = call(pool, nq, nk, qs, kk, vs, out=big[:, 1:, 8:8 + d])
        assert np.array_equal(bits(out), bits(ref)) and torch.equal(lse, lref)
    assert (big[:, 0] == 7).all() and (big[:, 1:, :8] == 7).all() and (big[:, 1:, 8 + d:] == 7).all()
    B.tf_prompt_attend(pool, nq, nk, q, k, v, d ** -0.5, out, ws=torch.empty(max(256, B.tf_prompt_workspace_bytes(nq, nk, H, Hkv, d, d)),
                                                                          dtype=torch.uint8, device="cuda"))   # without lse
    assert np.array_equal(bits(out), bits(ref))


def test_rows_behind_two_to_the_31(pool):
    """Keys whose values start past 2^31: the last stream's."""
    H, dqk, dv = 64, 192, 128
    nq, nk = [1, 130], [140000, 200]
    kv = torch.zeros((sum(nk), H, dqk - 64 + dv), dtype=torch.bfloat16, device="cuda")
    assert 140000 * H * (dqk - 64 + dv) > 2 ** 31
    q, k, v, kr = make([131], [200], H, H, dqk, dv, True, seed=13)
    kv[140000:, :, :dqk - 64], kv[140000:, :, dqk - 64:] = k, v
    krb = torch.zeros((sum(nk), 64), dtype=torch.bfloat16, device="cuda")
    krb[140000:] = kr
    out, lse = call(pool, nq, nk, q, kv[..., :dqk - 64], kv[..., dqk - 64:], kr=krb)
    check([130], [200], q[1:], k, v, kr, True, out[1:], lse[1:], rows=20)
    assert not out[0].any() and (lse[0] - np.log(140000)).abs().max() < 1e-4


@pytest.mark.parametrize("nq,nk,H,Hkv", [([1, 1], [9000, 700], 16, 2), ([900, 300, 77], [900, 2000, 77], 8, 8)])
def test_repeated_and_captured_calls_are_bit_identical(pool, nq, nk, H, Hkv):
    q, k, v, kr = make(nq, nk, H, Hkv, 192, 128, True, seed=14)
    ref, lref = call(pool, nq, nk, q, k, v, kr=kr)
    for _ in range(20):
        out, lse = call(pool, nq, nk, q, k, v, kr=kr)
        assert np.array_equal(bits(out), bits(ref)) and torch.equal(lse, lref)
    n = B.tf_prompt_workspace_bytes(nq, nk, H, Hkv, 192, 128)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    out, lse = torch.empty_like(ref), torch.empty_like(lref)
    with torch.cuda.graph(g, stream=side):
        B.tf_prompt_attend(pool, nq, nk, q, k, v, 192 ** -0.5, out, lse=lse, kr=kr, ws=ws)
    out.fill_(float("nan"))
    q2 = q.clone()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    no_device_error(pool)
    assert np.array_equal(bits(out), bits(ref)) and torch.equal(lse, lref)
    q.copy_(-q2)          # a replay reads what the tensors hold then
    g.replay()
    torch.cuda.synchronize()
    o2, _ = call(pool, nq, nk, -q2, k, v, kr=kr)
    assert np.array_equal(bits(out), bits(o2))


def test_calls_on_two_streams(pool):
    cases = [([700, 33], [700, 800], 8, 2, 1), ([1, 1, 1], [4000, 12000, 5], 16, 2, 2)]
    xs = [make(nq, nk, H, Hkv, 128, 128, seed=s) for nq, nk, H, Hkv, s in cases]
    refs = [call(pool, c[0], c[1], *x) for c, x in zip(cases, xs)]
    streams = [torch.cuda.Stream() for _ in cases]
    outs, ws = [], []
    for c, x in zip(cases, xs):
        n = B.tf_prompt_workspace_bytes(c[0], c[1], c[2], c[3], 128, 128)
        ws.append(torch.empty(max(n, 256), dtype=torch.uint8, device="cuda"))
        outs.append((torch.empty((sum(c[0]), c[2], 128), dtype=torch.bfloat16, device="cuda"), torch.empty((sum(c[0]), c[2]), device="cuda")))
    torch.cuda.synchronize()
    for _ in range(10):
        for st, c, x, o, w in zip(streams, cases, xs, outs, ws):
            B.tf_prompt_attend(pool, c[0], c[1], x[0], x[1], x[2], 128 ** -0.5, o[0], lse=o[1], ws=w, stream=st.cuda_stream)
    torch.cuda.synchronize()
    no_device_error(pool)
    for o, r in zip(outs, refs):
        assert np.array_equal(bits(o[0]), bits(r[0])) and torch.equal(o[1], r[1])
