"""GPU parity of rotary positions, the append of a projection's rows and the rows back from the pages, against the
fp64 definitions, through the C-ABI.

Tolerances.  u = 2^-8 is half a bf16 step (relative), f = 2^-24 half an fp32 step.  An angle is off by 0.16 2^-21 turns
at most for the frequency (three double roundings, times a position below 2^31 and at most 0.16 turns a position), by
2^-25 + 2^-32 turns as a fraction cut to fp32, and by two roundings of at most pi on its way into the sine: 1.03e-6
radians.  The hardware's sine and cosine add 2^-21.19 = 4.2e-7, the products and sums 4 f = 2.4e-7: a turned pair is off by less
than 1.7e-6 < 2^-18.5 = 2.7e-6 times A (|a| + |b|), and by its rounding u |ref|.
A norm's factor is off by (512 + 8) f relative (a sum of squares in any order), so a latent value by 2^-14 + u.
"""
import numpy as np
import pytest
import torch

from oracle import fp8 as F8
from oracle import prompt as O
from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from tests.gpu_common import bits, no_device_error

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
YARN = dict(scaling=B.TF_ROPE_YARN, factor=8.0, original=4096.0)
SCALINGS = {"plain": {}, "linear": dict(scaling=B.TF_ROPE_LINEAR, factor=4.0), "yarn": YARN}


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()
    B.lib()


def host(t):
    return t.double().cpu().numpy()


def randn(*s, seed=0):
    return torch.randn(s, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def freq(dim, name, base=10000.0):
    how = SCALINGS[name]
    return O.frequencies(dim, base, name, how.get("factor", 1.0), how.get("original", 0.0))


def positions(pos, n):
    return [p + i for p, k in zip(pos, n) for i in range(k)]


def check_turned(got, x, where, dim, name, half):
    f, amp = freq(dim, name)
    ref = O.rotate(x, where, f, amp, half)
    pairs = np.abs(x[..., :dim // 2]) + np.abs(x[..., dim // 2:]) if half else np.abs(x[..., 0::2]) + np.abs(x[..., 1::2])
    both = np.concatenate([pairs, pairs], -1) if half else np.repeat(pairs, 2, -1)
    assert np.all(np.abs(got - ref) <= 2.0 ** -18.5 * amp * both + U * np.abs(ref))


# ---- rotary positions ----------------------------------------------------------------------------

@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 128, 256])
@pytest.mark.parametrize("H", [1, 3, 16])
def test_rope_dims_and_heads(dim, H, half):
    pos, n = [0, 5000, 1 << 20, 7], [3, 0, 2, 6]
    rope = B.tf_rope_make(dim, layout=int(half))
    x = randn(11, H, dim, seed=dim)
    y = torch.full_like(x, float("nan"))
    B.tf_rope_apply(rope, pos, n, x, y)
    check_turned(host(y), host(x), positions(pos, n), dim, "plain", half)
    B.tf_rope_apply(rope, pos, n, x)                     # in place
    assert np.array_equal(bits(x), bits(y))


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("name", ["plain", "linear", "yarn"])
@pytest.mark.parametrize("pos", [0, 1000000, 2 ** 31 - 40])
def test_rope_scalings_and_far_positions(pos, name, half):
    rope = B.tf_rope_make(64, layout=int(half), **SCALINGS[name])
    x = randn(40, 2, 64, seed=3)
    y = torch.empty_like(x)
    B.tf_rope_apply(rope, [pos], [40], x, y)
    check_turned(host(y), host(x), range(pos, pos + 40), 64, name, half)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("rows,H,head", [(1, 64, 576), (64, 64, 576), (3001, 8, 192), (700, 128, 64), (5000, 1, 64)])
def test_rope_of_a_part_of_the_heads(rows, H, head, half):
    """The last 64 values of every head: the others stay, in both tensors."""
    n, left = [], rows
    while left:
        n.append(min(left, 1 + (37 * len(n)) % 911))
        left -= n[-1]
    pos = [(i * 7919) % 100000 for i in range(len(n))]
    rope = B.tf_rope_make(64, layout=int(half), **YARN)
    x = randn(rows, H, head, seed=rows)
    y = torch.full_like(x, 7.0)
    keep = x.clone()
    B.tf_rope_apply(rope, pos, n, x[..., -64:], y[..., -64:])
    assert torch.equal(x, keep) and (y[..., :-64] == 7).all()
    some = sorted({0, rows - 1, rows // 2, rows // 3})
    where = positions(pos, n)
    check_turned(host(y[some][..., -64:]), host(x[some][..., -64:]), [where[i] for i in some], 64, "yarn", half)
    z = torch.zeros((rows, H, 72), dtype=torch.bfloat16, device="cuda")     # other strides, the same bits
    B.tf_rope_apply(rope, pos, n, x[..., -64:], z[..., 8:])
    assert np.array_equal(bits(z[..., 8:]), bits(y[..., -64:])) and not z[..., :8].any()


def test_rope_is_a_rotation_of_relative_position():
    """Products of turned queries and keys depend on the distance alone, also far out."""
    rope = B.tf_rope_make(128, layout=B.TF_ROPE_HALF)
    q, k = randn(1, 1, 128, seed=1).expand(2, 1, 128).contiguous(), randn(1, 1, 128, seed=2).expand(2, 1, 128).contiguous()
    p = [100, 2 ** 30 + 100]
    B.tf_rope_apply(rope, p, [1, 1], q)
    B.tf_rope_apply(rope, [a - 33 for a in p], [1, 1], k)
    a, b = (host(q) * host(k)).sum(-1)[:, 0]
    scale = (np.abs(host(q)) * np.abs(host(k))).sum(-1).max()
    assert abs(a - b) <= scale * 4 * U


# ---- the append of a projection's rows -------------------------------------------------------------

def tables(pool, lens, extra=0):
    npg = [max(1, -(-n // 512)) for n in lens]
    t = torch.full((len(lens), max(npg) + extra), -1, dtype=torch.int32)
    for s, k in enumerate(npg):
        t[s, :k] = torch.from_numpy(pool.take(k))
    return t.cuda(), max(npg) + extra


def held(pool, cache=0):
    """(latent or codes, scales, rope) of a cache as host arrays [pages][512][..]."""
    raw = pool.bytes_view()[cache].cpu().numpy()
    if not pool.fp8:
        x = raw.view(np.uint16)
        return x[:, :512 * 512].reshape(-1, 512, 512), None, x[:, 512 * 512:].reshape(-1, 512, 64)
    return (raw[:, :262144].reshape(-1, 512, 512), raw[:, 262144:264192].copy().view(np.float32),
            raw[:, 264192:].copy().view(np.uint16).reshape(-1, 512, 64))


def values(b):
    return (np.asarray(b, np.uint32) << 16).view(np.float32).astype(np.float64)


def norm_ref(x, gain):
    return O.rms_norm(x, gain, 1e-6)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("norm,turn", [(True, True), (False, True), (True, False), (False, False)])
def test_append(fp8, half, norm, turn):
    pos, n = [0, 511, 3, 1000, 77], [600, 2, 0, 90, 1]
    pool = B.KVPool(2, 12, poison=True, seed=5, fp8=fp8)
    pt, mp = tables(pool, [a + b for a, b in zip(pos, n)])
    N = sum(n)
    big = randn(N, 640, seed=21)
    big[5, :512] = 0                                   # a row of zeros
    rows = big[:, :576]
    gain = (1 + 0.25 * torch.randn(512, device="cuda")).bfloat16() if norm else None
    rope = B.tf_rope_make(64, layout=int(half), **YARN) if turn else None
    before, other = held(pool, 1), pool.bytes_view()[0].clone()
    B.tf_paged_append_rope(pool, 1, pt, mp, pos, n, rows, gain=gain, eps=1e-6, rope=rope)
    no_device_error(pool)
    lat, scales, key = held(pool, 1)
    x = host(rows)
    table = pt.cpu().numpy()
    seen = np.zeros(lat.shape[:2], bool)
    j = 0
    for s, (p, k) in enumerate(zip(pos, n)):
        for i in range(k):
            page, r = table[s, (p + i) // 512], (p + i) % 512
            seen[page, r] = True
            y = norm_ref(x[j, :512], host(gain)) if norm else x[j, :512]
            if fp8:
                z = float(scales[page, r])
                amax = np.abs(y).max()
                assert abs(z - amax / 448) <= 2.0 ** -13 * amax / 448
                code = F8.decode_table()[lat[page, r]]
                # half a step of the code (2^-4 relative, 2^-10 below the smallest normal), of a value off by 2^-13
                assert np.all(np.abs(code * z - y) <= (2.0 ** -4 + 2.0 ** -12) * np.abs(y) + 2.0 ** -10 * z * (1 + 2.0 ** -12))
                if not norm:
                    c, sc = F8.quantize_row(x[j, :512].astype(np.float32))
                    assert np.array_equal(lat[page, r], c) and z == sc
            else:
                got = values(lat[page, r])
                assert np.all(np.abs(got - y) <= (U + 2.0 ** -13 if norm else 0) * np.abs(y))
            if turn:
                check_turned(values(key[page, r])[None, None], x[j:j + 1, None, 512:], [p + i], 64, "yarn", half)
            else:
                assert np.array_equal(values(key[page, r]), x[j, 512:])
            j += 1
    for a, b in zip((lat, key) if not fp8 else (lat, scales, key), (before[0], before[2]) if not fp8 else before):
        assert np.array_equal(np.asarray(a)[~seen].view(np.uint8), np.asarray(b)[~seen].view(np.uint8))   # nothing else was written
    assert torch.equal(pool.bytes_view()[0], other)      # nor another cache


@pytest.mark.parametrize("fp8", [False, True])
def test_plain_append_equals_the_append(fp8):
    """Without norm and rotation: tf_paged_append's bits."""
    pos, n = [500, 0], 40
    a, b = (B.KVPool(1, 6, poison=True, fp8=fp8) for _ in range(2))
    (pa, mp), (pb, _) = tables(a, [540, 40]), tables(b, [540, 40])
    assert torch.equal(pa, pb)
    rows = randn(2 * n, 576, seed=4)
    B.tf_paged_append(a, 0, pa, mp, pos, rows[:, :512].contiguous().view(2, n, 512), rows[:, 512:].contiguous().view(2, n, 64))
    B.tf_paged_append_rope(b, 0, pb, mp, pos, [n, n], rows)
    assert sorted(pa.unique().tolist()) == [-1, 0, 1, 2]           # the pages that were taken, and poisoned
    assert torch.equal(a.bytes_view()[:, :3], b.bytes_view()[:, :3])


@pytest.mark.parametrize("fp8", [False, True])
def test_windows_without_a_table(fp8):
    pool = B.KVPool(1, 6, poison=True, fp8=fp8)
    pool.take(6)
    rows = randn(700, 576, seed=6)
    B.tf_paged_append_rope(pool, 0, None, 3, [900, 0], [600, 100], rows)
    lat, key = torch.empty((700, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((700, 64), dtype=torch.bfloat16, device="cuda")
    B.tf_paged_read(pool, 0, None, 3, [900, 0], [600, 100], latent=lat, rope=key)
    no_device_error(pool)
    assert np.array_equal(bits(key), bits(rows[:, 512:]))
    if not fp8:
        assert np.array_equal(bits(lat), bits(rows[:, :512]))
    other = torch.empty_like(lat)
    B.tf_paged_read(pool, 0, torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3), 3, [900, 0], [600, 100], latent=other)
    assert np.array_equal(bits(lat), bits(other))


def test_norm_of_large_and_small_rows():
    """Square sums near fp32's ends, and rows far below eps."""
    pool = B.KVPool(1, 1)
    pt, mp = tables(pool, [8])
    x = randn(4, 576, seed=8)
    x = x * torch.tensor([1e-12, 1e-3, 1.0, 1e17], device="cuda")[:, None].bfloat16()
    gain = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    B.tf_paged_append_rope(pool, 0, pt, mp, [0], [4], x, gain=gain, eps=1e-6)
    lat, _, _ = held(pool)
    page = int(pt[0, 0])
    for i in range(4):
        y = norm_ref(host(x)[i, :512], np.ones(512))
        assert np.all(np.abs(values(lat[page, i]) - y) <= (U + 2.0 ** -13) * np.abs(y) + 2.0 ** -133)


# ---- rows back from the pages ------------------------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("start,n", [([0], [1]), ([511], [2]), ([1, 1300, 0, 9], [1100, 37, 0, 512])])
def test_read(start, n, fp8):
    pool = B.KVPool(3, 16, poison=True, seed=9, fp8=fp8)
    lens = [a + b for a, b in zip(start, n)]
    pt, mp = tables(pool, lens, extra=1)
    rows = randn(sum(lens), 576, seed=10)
    B.tf_paged_append_rope(pool, 2, pt, mp, [0] * len(n), lens, rows)
    N = sum(n)
    both = torch.full((N + 1, 640), 7.0, dtype=torch.bfloat16, device="cuda")
    B.tf_paged_read(pool, 2, pt, mp, start, n, latent=both[:N, :512], rope=both[:N, 520:584])
    no_device_error(pool)
    off = np.cumsum([0] + lens)
    at = np.concatenate([np.arange(o + a, o + a + k) for o, a, k in zip(off, start, n)])
    want = rows[torch.from_numpy(at).cuda()]
    assert np.array_equal(bits(both[:N, 520:584]), bits(want[:, 512:]))
    if fp8:
        x = F8.dequantize_rows(*F8.quantize_rows(want[:, :512].float().cpu().numpy()))
        assert np.array_equal(bits(both[:N, :512]), bits(torch.from_numpy(x.astype(np.float32)).bfloat16()))
    else:
        assert np.array_equal(bits(both[:N, :512]), bits(want[:, :512]))
    assert (both[:N, 512:520] == 7).all() and (both[:, 584:] == 7).all() and (both[N] == 7).all()
    only = torch.empty((N, 64), dtype=torch.bfloat16, device="cuda")
    B.tf_paged_read(pool, 2, pt, mp, start, n, rope=only)
    assert np.array_equal(bits(only), bits(want[:, 512:]))
    only = torch.empty((N, 512), dtype=torch.bfloat16, device="cuda")
    B.tf_paged_read(pool, 2, pt, mp, start, n, latent=only)
    assert np.array_equal(bits(only), bits(both[:N, :512]))


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_pages_are_recorded_and_skipped(fp8):
    pool = B.KVPool(1, 4, poison=True, fp8=fp8)
    pt, mp = tables(pool, [600, 600])
    rows = randn(1200, 576, seed=12)
    bad = pt.clone()
    bad[0, 1], bad[1, 0] = 4, -3
    B.tf_paged_append_rope(pool, 0, bad, mp, [0, 0], [600, 600], rows)
    rc, detail = pool.last_error()
    assert rc == B.TF_E_DEVICE and detail in (4, -3)
    B.tf_paged_append_rope(pool, 0, pt, mp, [0, 0], [600, 600], rows)
    lat, key = torch.full((1200, 512), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((1200, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    B.tf_paged_read(pool, 0, bad, mp, [0, 0], [600, 600], latent=lat, rope=key)
    rc, detail = pool.last_error()
    assert rc == B.TF_E_DEVICE and detail in (4, -3)
    hit = torch.zeros(1200, dtype=torch.bool)
    hit[:512], hit[600 + 512:] = True, True
    assert np.array_equal(bits(key[hit]), bits(rows[hit][:, 512:])) and (key[~hit] == 7).all() and (lat[~hit] == 7).all()
    unread = pt.clone()
    unread[0, 1] = 99                                    # of a page that the call does not read
    B.tf_paged_read(pool, 0, unread, mp, [0, 0], [512, 600], latent=lat[:1112], rope=key[:1112])
    no_device_error(pool)


# ---- together ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True])
def test_append_decode_and_prompt_agree(fp8):
    """A layer as a model runs it: prompts are written, read back, projected and attended with heads of their own; the
    absorbed attention over the same pages gives the same outputs, up to its roundings."""
    H, dn, dv = 16, 128, 128
    lens = [700, 33, 129]
    pool = B.KVPool(1, 8, poison=True, fp8=fp8)
    pt, mp = tables(pool, lens)
    N = sum(lens)
    rows, gain = randn(N, 576, seed=30), (1 + 0.1 * torch.randn(512, device="cuda")).bfloat16()
    rope = B.tf_rope_make(64)
    B.tf_paged_append_rope(pool, 0, pt, mp, [0] * 3, lens, rows, gain=gain, rope=rope)
    lat, key = torch.empty((N, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((N, 64), dtype=torch.bfloat16, device="cuda")
    B.tf_paged_read(pool, 0, pt, mp, [0] * 3, lens, latent=lat, rope=key)
    wk, wv = randn(H, dn, 512, seed=31) * 512 ** -0.5, randn(H, dv, 512, seed=32) * 512 ** -0.5
    kv = torch.cat([torch.einsum("nc,hdc->nhd", lat.float(), wk.float()), torch.einsum("nc,hdc->nhd", lat.float(), wv.float())], -1).bfloat16()
    q = randn(N, H, dn + 64, seed=33)
    B.tf_rope_apply(rope, [0] * 3, lens, q[..., dn:])
    out = torch.empty((N, H, dv), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((N, H), device="cuda")
    n = B.tf_prompt_workspace_bytes(lens, lens, H, H, dn + 64, dv)
    scale = (dn + 64) ** -0.5
    B.tf_prompt_attend(pool, lens, lens, q, kv[..., :dn], kv[..., dn:], scale, out, lse=lse, kr=key,
                       ws=torch.empty(n, dtype=torch.uint8, device="cuda") if n else None)
    # the last token of each prompt, absorbed
    last = torch.tensor(np.cumsum(lens) - 1).cuda()
    qa = torch.cat([torch.einsum("shd,hdc->shc", q[last][..., :dn].float(), wk.float()).bfloat16(), q[last][..., dn:]], -1)[:, None].contiguous()
    oa = torch.empty((3, 1, H, 512), dtype=torch.bfloat16, device="cuda")
    la = torch.empty((3, 1, H), device="cuda")
    n = B.tf_paged_mla_workspace_bytes(pool, 3, 1, H, lens)
    B.tf_paged_mla_attend(pool, 0, pt, mp, lens, qa, scale, oa, la, ws=torch.empty(n, dtype=torch.uint8, device="cuda") if n else None)
    no_device_error(pool)
    proj = torch.einsum("shc,hdc->shd", oa[:, 0].float(), wv.float())
    # queries, keys and values are rounded at other places: relative 2^-8 each on the way to a score and to an output
    assert ((proj - out[last].float()).norm() / proj.norm()).item() <= 6 * U
    assert (la[:, 0] - lse[last]).abs().max().item() <= 6 * U * 4


def test_a_layer_captured_as_one_graph():
    """Append, rotation and attention of a decode step in one graph, replayed after the rows changed."""
    H, S = 16, 4
    lens = [512, 100, 1025, 7]
    pool = B.KVPool(1, 16, poison=True)
    pt, mp = tables(pool, lens)
    rope = B.tf_rope_make(64, layout=B.TF_ROPE_HALF)
    gain = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    B.tf_paged_append_rope(pool, 0, pt, mp, [0] * S, lens, randn(sum(lens), 576, seed=40), gain=gain, rope=rope)
    new, q = randn(S, 576, seed=41), randn(S, 1, H, 576, seed=42)
    qt = torch.empty_like(q)
    out = torch.empty((S, 1, H, 512), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(256, B.tf_paged_mla_workspace_bytes(pool, S, 1, H, lens)), dtype=torch.uint8, device="cuda")
    last = [n - 1 for n in lens]

    def step():
        B.tf_paged_append_rope(pool, 0, pt, mp, last, [1] * S, new, gain=gain, rope=rope)
        qt[..., :512].copy_(q[..., :512])
        B.tf_rope_apply(rope, last, [1] * S, q[:, 0, :, 512:], qt[:, 0, :, 512:])
        B.tf_paged_mla_attend(pool, 0, pt, mp, lens, qt, 576 ** -0.5, out, ws=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (50, 51):
        new.copy_(randn(S, 576, seed=seed))
        q.copy_(randn(S, 1, H, 576, seed=seed + 10))
        step()
        want = out.clone()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits(out), bits(want))
    no_device_error(pool)


@pytest.mark.parametrize("fp8", [False, True])
def test_launch_timing_covers_the_calls(fp8):
    pool = B.KVPool(1, 4, fp8=fp8)
    pt, mp = tables(pool, [300])
    pool.profile(True)
    rows = randn(300, 576, seed=60)
    B.tf_paged_append_rope(pool, 0, pt, mp, [0], [300], rows)
    lat = torch.empty((300, 512), dtype=torch.bfloat16, device="cuda")
    B.tf_paged_read(pool, 0, pt, mp, [0], [300], latent=lat)
    q, k, v = randn(300, 2, 64, seed=61), randn(300, 2, 64, seed=62), randn(300, 2, 64, seed=63)
    out = torch.empty_like(q)
    n = B.tf_prompt_workspace_bytes([300], [300], 2, 2, 64, 64)
    B.tf_prompt_attend(pool, [300], [300], q, k, v, 0.125, out, ws=torch.empty(n, dtype=torch.uint8, device="cuda") if n else None)
    for kind in (B.PROF_APPEND, B.PROF_COPY, B.PROF_ATTEND):
        ms, count = pool.profile_read(kind)
        assert count == 1 and 0 < ms < 50


def test_codes_equal_the_appends_at_every_magnitude():
    """FP8 codes and scales, bit for bit tf_paged_append's (whose quotients are IEEE divisions): rows from the smallest
    bf16 values to the largest, random bits, ties and mixed magnitudes."""
    g = torch.Generator(device="cuda").manual_seed(70)
    rows = []
    for e in range(-133, 128, 3):
        rows.append(torch.randn((4, 576), generator=g, device="cuda").double() * 2.0 ** e)
    rows.append(torch.randn((300, 576), generator=g, device="cuda").double() * 2.0 ** torch.randint(-60, 60, (300, 576), generator=g, device="cuda").double())
    ties = torch.arange(576, device="cuda").double() / 16          # quotients half way between codes
    rows.append(torch.stack([ties * 448 / ties[:512].max(), ties, ties * 3, -ties * 7]))
    x = torch.cat(rows).clamp(-3.3e38, 3.3e38).bfloat16()
    x = torch.cat([x, torch.randint(0, 0x7F80, (500, 576), generator=g, device="cuda").to(torch.int16).view(torch.bfloat16)])
    n = x.shape[0]
    a, b = (B.KVPool(1, 8, poison=True, fp8=True) for _ in range(2))
    (pa, mp), (pb, _) = tables(a, [n]), tables(b, [n])
    B.tf_paged_append(a, 0, pa, mp, [0], x[:, :512].contiguous().view(1, n, 512), x[:, 512:].contiguous().view(1, n, 64))
    B.tf_paged_append_rope(b, 0, pb, mp, [0], [n], x)
    no_device_error(b)
    k = -(-n // 512)
    assert torch.equal(a.bytes_view()[:, :k], b.bytes_view()[:, :k])
