"""Host side of the prompt path: the rotary table, what the calls refuse before any launch, the work plan and the
workspace's size.  No GPU: the pool is made over an address that is never read."""
import ctypes
import math
import os
import shutil
import subprocess
import types

import numpy as np
import pytest
import torch

from oracle import prompt as O
from paged_mla_kv_gb300 import binding as B
from paged_mla_kv_gb300 import build as BUILD
from tests.test_host_block_devices import On
from tests.test_out_of_memory import HOST, preload, run   # noqa: F401 (a fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def L():
    BUILD.build()
    return B.lib()


def _pool(pages=32, caches=2, fp8=False):
    d = B.make_desc(caches, pages, fp8=fp8)
    h = ctypes.c_void_p()
    assert B.lib().tf_kvpool_create(ctypes.byref(d), ctypes.c_void_p(BASE), B.tf_kvpool_bytes(d), ctypes.byref(h)) == 0
    return h


keep = []


def i64(*a):
    a = np.asarray(a, np.int64)
    keep.append(a)
    return a.ctypes.data


# ---- the rotary table --------------------------------------------------------------------------------

@pytest.mark.parametrize("dim", [16, 64, 128, 256])
@pytest.mark.parametrize("name,how", [("plain", {}), ("linear", dict(scaling=B.TF_ROPE_LINEAR, factor=4.0)),
                                      ("yarn", dict(scaling=B.TF_ROPE_YARN, factor=8.0, original=4096.0)),
                                      ("yarn", dict(scaling=B.TF_ROPE_YARN, factor=40.0, original=65536.0, beta_fast=16.0, beta_slow=2.0))])
@pytest.mark.parametrize("base", [10000.0, 8e6])
def test_table_equals_the_oracles(dim, name, how, base):
    r = B.tf_rope_make(dim, base=base, **how)
    f, a = O.frequencies(dim, base, name, how.get("factor", 1.0), how.get("original", 0.0), how.get("beta_fast", 32.0),
                         how.get("beta_slow", 1.0))
    assert r.amplitude == np.float32(a) and r.dim == dim
    got = np.array([r.turn[i] for i in range(dim // 2)], np.float64) * 2.0 ** -64 * 2 * math.pi
    # pow, logarithms and five more double roundings on either side
    assert np.all(np.abs(got - f) <= 2.0 ** -48 * f + 2.0 ** -62)
    assert all(r.turn[i] == 0 for i in range(dim // 2, 128))
    assert B.tf_rope_make(dim, base=base, amplitude=0.75, **how).amplitude == 0.75


@pytest.mark.parametrize("bad", [dict(dim=8), dict(dim=24), dict(dim=272), dict(dim=0), dict(layout=2), dict(base=1.0), dict(base=float("nan")),
                                 dict(base=float("inf")), dict(scaling=3), dict(scaling=1, factor=0.5), dict(scaling=1, factor=float("inf")),
                                 dict(scaling=2, factor=2.0), dict(scaling=2, factor=2.0, original=4096.0, beta_slow=0.0),
                                 dict(scaling=2, factor=2.0, original=4096.0, beta_fast=1.0, beta_slow=1.0),
                                 dict(scaling=2, factor=2.0, original=4096.0, beta_fast=float("inf")), dict(amplitude=-1.0),
                                 dict(amplitude=1e300), dict(amplitude=float("nan"))])
def test_table_refusals(bad):
    with pytest.raises(B.TFError) as e:
        B.tf_rope_make(**dict(dict(dim=64), **bad))
    assert e.value.code == B.TF_E_ARG


def test_table_of_a_null_pointer(L):
    d, r = B.tf_rope_desc(64, 0, 0, 0, 10000.0, 1, 0, 32, 1, 0), B.tf_rope()
    assert L.tf_rope_make(None, ctypes.byref(r)) == B.TF_E_ARG and L.tf_rope_make(ctypes.byref(d), None) == B.TF_E_ARG
    d.reserved = 1
    assert L.tf_rope_make(ctypes.byref(d), ctypes.byref(r)) == B.TF_E_ARG


# ---- what the calls refuse ---------------------------------------------------------------------------

def test_rope_refusals(L):
    ropes = [B.tf_rope_make(64), B.tf_rope()]

    def call(rope=ropes[0], pos=(0, 5), n=(3, 4), S=2, H=16, x=BASE, xr=1024, xh=64, y=BASE, yr=1024, yh=64):
        return L.tf_rope_apply(ctypes.addressof(rope) if rope else None, i64(*pos), i64(*n), S, H, x, xr, xh, y, yr, yh, None)

    assert call(rope=None) == B.TF_E_ARG and call(rope=ropes[1]) == B.TF_E_ARG      # never made
    assert call(S=0) == B.TF_E_ARG and call(S=513) == B.TF_E_ARG
    assert call(H=0) == B.TF_E_ARG and call(H=129) == B.TF_E_ARG
    assert call(n=(3, -1)) == B.TF_E_ARG
    assert call(x=None) == B.TF_E_ARG and call(y=None) == B.TF_E_ARG
    assert call(x=BASE + 8) == B.TF_E_ARG and call(y=BASE + 2) == B.TF_E_ARG
    for k in ("xr", "xh", "yr", "yh"):
        assert call(**{k: 1028}) == B.TF_E_ARG
    assert call(pos=(0, -1)) == B.TF_E_RANGE and call(pos=(0, 2 ** 31 - 3)) == B.TF_E_RANGE
    assert call(pos=(0, 0), n=(2 ** 31, 0)) == B.TF_E_UNSUPPORTED
    assert call(pos=(0, 0), n=(2 ** 31 - 1, 1)) == B.TF_E_UNSUPPORTED
    assert call(n=(0, 0), x=None, y=None) == B.TF_OK                                # no rows: nothing is launched
    assert L.tf_rope_apply(ctypes.addressof(ropes[0]), None, i64(1), 1, 1, BASE, 64, 64, BASE, 64, 64, None) == B.TF_E_ARG
    assert L.tf_rope_apply(ctypes.addressof(ropes[0]), i64(1), None, 1, 1, BASE, 64, 64, BASE, 64, 64, None) == B.TF_E_ARG


@pytest.mark.parametrize("fp8", [False, True])
def test_append_refusals(L, fp8):
    h = _pool(fp8=fp8)
    ropes = [B.tf_rope_make(64), B.tf_rope_make(128), B.tf_rope()]

    def call(pool=h, cache=0, pt=BASE, mp=4, pos=(100, 2000), n=(5, 48), S=2, rows=BASE, stride=576, gain=BASE, eps=1e-6, rope=ropes[0]):
        return L.tf_paged_append_rope(pool, cache, pt, mp, i64(*pos), i64(*n), S, rows, stride, gain, eps,
                                      ctypes.addressof(rope) if rope else None, None)

    assert call(pool=None) == B.TF_E_ARG and call(rows=None) == B.TF_E_ARG and call(rows=BASE + 8) == B.TF_E_ARG
    assert call(S=0) == B.TF_E_ARG and call(S=513) == B.TF_E_ARG and call(mp=0) == B.TF_E_ARG and call(n=(1, -1)) == B.TF_E_ARG
    assert call(stride=575) == B.TF_E_ARG and call(stride=568) == B.TF_E_ARG and call(stride=580) == B.TF_E_ARG
    assert call(gain=BASE + 4) == B.TF_E_ARG
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert call(eps=eps) == B.TF_E_ARG
    assert call(rope=ropes[1]) == B.TF_E_ARG and call(rope=ropes[2]) == B.TF_E_ARG
    assert call(cache=2) == B.TF_E_RANGE and call(cache=-1) == B.TF_E_RANGE
    assert call(pos=(100, 2001)) == B.TF_E_RANGE and call(pos=(-1, 0)) == B.TF_E_RANGE
    assert call(pt=None, mp=17, pos=(0, 0)) == B.TF_E_RANGE
    assert call(mp=1 << 30, pos=(0, 2 ** 31 - 10)) == B.TF_E_RANGE                   # past the last position
    assert call(mp=1 << 30, pos=(0, 0), n=(2 ** 31 - 1, 1)) == B.TF_E_UNSUPPORTED
    assert call(n=(0, 0), rows=None) == B.TF_OK
    assert call(gain=None, eps=0.0, n=(0, 0)) == B.TF_OK                             # no norm: eps is not read


def test_read_refusals(L):
    h = _pool()

    def call(pool=h, cache=0, pt=BASE, mp=4, start=(100, 2000), n=(5, 48), S=2, lat=BASE, ls=512, rope=BASE, rs=64):
        return L.tf_paged_read(pool, cache, pt, mp, i64(*start), i64(*n), S, lat, ls, rope, rs, None)

    assert call(pool=None) == B.TF_E_ARG and call(lat=None, rope=None) == B.TF_E_ARG
    assert call(lat=BASE + 8) == B.TF_E_ARG and call(rope=BASE + 8) == B.TF_E_ARG
    assert call(ls=504) == B.TF_E_ARG and call(ls=516) == B.TF_E_ARG and call(rs=56) == B.TF_E_ARG and call(rs=68) == B.TF_E_ARG
    assert call(S=0) == B.TF_E_ARG and call(S=513) == B.TF_E_ARG and call(mp=0) == B.TF_E_ARG and call(n=(1, -1)) == B.TF_E_ARG
    assert call(cache=2) == B.TF_E_RANGE and call(start=(100, 2001)) == B.TF_E_RANGE and call(start=(-1, 0)) == B.TF_E_RANGE
    assert call(pt=None, mp=17) == B.TF_E_RANGE
    assert call(n=(0, 0)) == B.TF_OK and call(n=(0, 0), lat=None, ls=0) == B.TF_OK and call(n=(0, 0), rope=None, rs=0) == B.TF_OK


def heads(p=BASE, row=1024, head=128):
    x = B.tf_heads(p, row, head)
    keep.append(x)
    return ctypes.addressof(x)


def test_attend_refusals(L):
    h = _pool()

    def call(pool=h, nq=(3, 40), nk=(3, 100), S=2, H=8, Hkv=4, dqk=192, dv=128, q=heads(), k=heads(), kr=BASE, kr_row=64, v=heads(), scale=0.1,
             causal=1, out=heads(), lse=None, ws=None, wsb=0):
        return L.tf_prompt_attend(pool, i64(*nq), i64(*nk), S, H, Hkv, dqk, dv, q, k, kr, kr_row, v, scale, causal, out, lse, ws, wsb, None)

    assert call(pool=None) == B.TF_E_ARG
    for name in ("q", "k", "v", "out"):
        assert call(**{name: None}) == B.TF_E_ARG and call(**{name: heads(p=0)}) == B.TF_E_ARG
        assert call(**{name: heads(p=BASE + 8)}) == B.TF_E_ARG and call(**{name: heads(row=1020)}) == B.TF_E_ARG
        assert call(**{name: heads(head=4)}) == B.TF_E_ARG
        if name != "out":
            assert call(**{name: heads(row=0)}) == B.TF_E_ARG and call(**{name: heads(row=-1024)}) == B.TF_E_ARG
            assert call(**{name: heads(head=0)}) == B.TF_E_ARG and call(**{name: heads(row=1 << 37)}) == B.TF_E_ARG
    assert call(kr=BASE + 2) == B.TF_E_ARG and call(kr_row=4) == B.TF_E_ARG and call(kr_row=0) == B.TF_E_ARG
    assert call(S=0) == B.TF_E_ARG and call(S=513) == B.TF_E_ARG
    assert call(H=0) == B.TF_E_ARG and call(H=129) == B.TF_E_ARG and call(Hkv=0) == B.TF_E_ARG and call(Hkv=3) == B.TF_E_ARG
    assert call(nq=(3, -1)) == B.TF_E_ARG and call(nk=(-1, 3)) == B.TF_E_ARG
    for scale in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert call(scale=scale) == B.TF_E_ARG
    assert call(causal=2) == B.TF_E_ARG and call(causal=-1) == B.TF_E_ARG
    for d in ((64, 128), (128, 64), (192, 192), (256, 128), (0, 0)):
        assert call(dqk=d[0], dv=d[1], kr=None) == B.TF_E_UNSUPPORTED
    assert call(dqk=64, dv=64) == B.TF_E_UNSUPPORTED                                 # a rotary key beside 64 values
    assert call(nq=(2 ** 31 - 1, 1)) == B.TF_E_UNSUPPORTED and call(nk=(2 ** 31 - 1, 1)) == B.TF_E_UNSUPPORTED
    assert call(nq=(0, 0), q=heads(p=0), out=heads(p=0)) == B.TF_OK                   # no rows
    n = B.tf_prompt_workspace_bytes([1], [40000], 8, 4, 192, 128)
    assert n > 0
    one = dict(nq=(1,), nk=(40000,), S=1)
    assert call(**one) == B.TF_E_ARG and call(ws=BASE, wsb=n - 1, **one) == B.TF_E_NOMEM and call(ws=BASE + 16, wsb=n + 16, **one) == B.TF_E_ARG


def test_sizes_and_plans_of_refused_calls(L):
    for a in (([3], [-1], 4, 4, 128, 128), ([3], [3], 4, 3, 128, 128), ([3], [3], 0, 1, 128, 128), ([3], [3], 4, 4, 128, 64), ([], [], 4, 4, 128, 128)):
        assert B.tf_prompt_workspace_bytes(*a) == 0
        with pytest.raises(B.TFError):
            B.tf_prompt_plan_info(*a)
    assert L.tf_prompt_plan_info(i64(1), i64(1), 1, 1, 1, 128, 128, 1, 0, None) == B.TF_E_ARG
    for f in (B.tf_prompt_workspace_bytes, B.tf_prompt_plan_info):
        with pytest.raises(B.TFError):
            f([1, 2], [1], 4, 4, 128, 128)


# ---- the plan ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("sms", [1, 7, 152, 240])
def test_plan(sms):
    """Every block of every stream is there as often as its keys are split; no split, no partials."""
    r = np.random.default_rng(6)
    for _ in range(300):
        S = int(r.integers(1, 20))
        Hkv = int(r.choice([1, 2, 8, 64]))
        G = int(r.choice([g for g in (1, 2, 3, 5, 8, 64, 128) if g * Hkv <= 128]))
        nq = [int(x) for x in r.integers(0, 2, S) * r.integers(0, 10 ** int(r.integers(1, 5)), S)]
        nk = [int(n + x) for n, x in zip(nq, r.integers(0, 10 ** int(r.integers(1, 6)), S))]
        d = [(64, 64), (128, 128), (192, 128)][int(r.integers(0, 3))]
        p = B.tf_prompt_plan_info(nq, nk, Hkv * G, Hkv, *d, causal=bool(r.integers(0, 2)), sms=sms)
        tpt = 128 // G
        blocks = [-(-n // (2 * tpt)) for n in nq]
        assert p["rows"] == 2 * tpt * G
        assert p["items"] >= sum(blocks) * Hkv
        assert (p["slots"] == 0) == (p["splits"] == 1)
        if p["splits"] == 1:
            assert p["items"] == sum(blocks) * Hkv
        else:
            tiles = max(-(-k // 128) for n, k in zip(nq, nk) if n)
            assert p["splits"] <= tiles and p["slots"] <= 2 * p["items"] and p["slots"] % 2 == 0
            assert p["items"] <= 40 * sms + sum(blocks) * Hkv


def test_workspace_holds_the_plans_slots():
    """Without a GPU sizes are those of 240 SMs, as the plans of 240 are."""
    if torch.cuda.is_available():
        pytest.skip("the current device decides")
    for nq, nk, H, Hkv, d in [([1], [100000], 8, 8, (128, 128)), ([1] * 16, [60000] * 16, 64, 8, (192, 128)), ([2], [5000], 4, 1, (64, 64)), ([300], [300], 4, 4, (64, 64))]:
        p = B.tf_prompt_plan_info(nq, nk, H, Hkv, *d, sms=240)
        n = p["slots"] * 128 * (d[1] * 4 + 8)
        assert B.tf_prompt_workspace_bytes(nq, nk, H, Hkv, *d) == -(-n // 256) * 256


# ---- the binding -------------------------------------------------------------------------------------

BF = dict(dtype=torch.bfloat16)


def calls():
    pool = types.SimpleNamespace(handle=None, num_pages=4, device=0)   # a null handle: nothing can be launched
    t = {"pt": torch.zeros(2, 2, dtype=torch.int32), "rows": torch.zeros(5, 576, **BF), "gain": torch.zeros(512, **BF),
         "latent": torch.zeros(5, 512, **BF), "rope": torch.zeros(5, 64, **BF), "q": torch.zeros(5, 4, 192, **BF),
         "k": torch.zeros(7, 2, 128, **BF), "v": torch.zeros(7, 2, 128, **BF), "kr": torch.zeros(7, 64, **BF),
         "out": torch.zeros(5, 4, 128, **BF), "lse": torch.zeros(5, 4), "ws": torch.zeros(256, dtype=torch.uint8)}
    return {
        "append": (lambda a: B.tf_paged_append_rope(pool, 0, a["pt"], 2, [0, 0], [2, 3], a["rows"], gain=a["gain"], rope=B.tf_rope_make(64), stream=0),
                   {k: t[k] for k in ("pt", "rows", "gain")}),
        "read": (lambda a: B.tf_paged_read(pool, 0, a["pt"], 2, [0, 0], [2, 3], latent=a["latent"], rope=a["rope"], stream=0),
                 {k: t[k] for k in ("pt", "latent", "rope")}),
        "attend": (lambda a: B.tf_prompt_attend(pool, [2, 3], [4, 3], a["q"], a["k"], a["v"], 0.1, a["out"], lse=a["lse"], kr=a["kr"],
                                                ws=a["ws"], stream=0), {k: t[k] for k in ("q", "k", "v", "kr", "out", "lse", "ws")})}


CASES = [(c, t) for c, (_, ts) in calls().items() for t in ts]


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
    assert e.value.code == B.TF_E_ARG and "device" not in str(e.value) and "form" not in str(e.value)


@pytest.mark.parametrize("call,tensor", [c for c in CASES if c[1] != "ws"])
def test_wrong_forms_are_refused(call, tensor):
    f, ts = calls()[call]
    t = ts[tensor]
    wrong = [t.to(torch.float64), t[:-1]]
    if t.dim() > 1:
        wrong += [torch.cat([t, t], -1), torch.cat([t, t], -1)[..., ::2]] if tensor != "pt" else []
    if tensor == "pt":
        wrong = [t.long(), t[:1], torch.zeros(2, 4, dtype=torch.int32)[:, ::2]]
    for w in wrong:
        args = {k: On(v, 0) for k, v in ts.items()}
        args[tensor] = On(w, 0)
        with pytest.raises(B.TFError) as e:
            f(args)
        assert e.value.code == B.TF_E_ARG and "form" in str(e.value), (tensor, tuple(w.shape))


def test_rope_forms():
    rope = B.tf_rope_make(64)
    x = torch.zeros(5, 4, 192, **BF)
    for xs, ys, pos, n in [(x, None, [0], [5]), (x[..., :64], x[..., :64].float(), [0], [5]), (x[..., :64], None, [0], [4]),
                           (x[..., :64], None, [0, 0], [5]), (x[..., :128:2], None, [0], [5]), (x[..., :64], x[:4, :, :64], [0], [5])]:
        with pytest.raises(B.TFError) as e:
            B.tf_rope_apply(rope, pos, n, On(xs, 0), None if ys is None else On(ys, 0), stream=0)
        assert e.value.code == B.TF_E_ARG and "form" in str(e.value)
    for a, b in [("host", "host"), (0, "host"), (0, 1), ("host", 0)]:
        put = lambda t, d: t if d == "host" else On(t, d)
        with pytest.raises(B.TFError) as e:
            B.tf_rope_apply(rope, [0], [5], put(x[..., :64], a), put(x[..., 64:128], b), stream=0)
        assert e.value.code == B.TF_E_ARG and "one GPU" in str(e.value)


def test_strides_of_single_rows_and_heads():
    """A tensor of one row or head may have any stride there; the library gets one that it takes."""
    x = torch.zeros(1, 1, 64, **BF).as_strided((1, 1, 64), (3, 5, 1))
    assert B._strides(x, (1, 1, 64), torch.bfloat16, "x") == (64, 64)
    assert B._row_stride(torch.zeros(1, 576, **BF).as_strided((1, 576), (7, 1)), 1, 576, torch.bfloat16, "x") == 576


# ---- host memory, the header -------------------------------------------------------------------------

OOM = {"size": "L.tf_prompt_workspace_bytes(n1, n1, 1, 64, 64, 192, 128, 1)",
       "plan": "L.tf_prompt_plan_info(n1, n1, 1, 64, 64, 192, 128, 1, 0, ctypes.byref(B.tf_prompt_plan()))",
       "attend": "L.tf_prompt_attend(plain, n1, n1, 1, 64, 64, 192, 128, h4, h4, None, 0, h4, 0.1, 1, h4, None, BASE, W, None)"}


@pytest.mark.parametrize("call", list(OOM))
def test_no_exception_leaves_a_call(preload, call):   # noqa: F811
    code = HOST + f"x4 = B.tf_heads(BASE, 24576, 192)\nh4 = ctypes.addressof(x4)\nfail(0)\nrc = {OOM[call]}\nfail(1 << 63)\nprint('rc', rc, B.TF_E_NOMEM)\n"
    r = run(code, preload)
    assert r.returncode == 0, r.stderr[-500:]
    rc, nomem = map(int, r.stdout.split()[1:])
    assert rc == (0 if call == "size" else nomem)


def test_header_is_c99_and_layouts_agree(tmp_path):
    src, exe = tmp_path / "a.c", tmp_path / "a"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "tf_prompt.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu %zu %zu\\n", sizeof(tf_rope_desc), sizeof(tf_rope), offsetof(tf_rope, turn), sizeof(tf_heads),'
                   ' sizeof(tf_prompt_plan), offsetof(tf_prompt_plan, rows));\nreturn 0; }\n')
    subprocess.run([shutil.which("gcc") or "gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", str(exe)], check=True)
    got = list(map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()))
    assert got == [ctypes.sizeof(B.tf_rope_desc), ctypes.sizeof(B.tf_rope), B.tf_rope.turn.offset, ctypes.sizeof(B.tf_heads),
                   ctypes.sizeof(B.tf_prompt_plan), B.tf_prompt_plan.rows.offset]
