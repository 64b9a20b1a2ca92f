"""Cases of the block-sparse and shared-prefix operators over a paged latent (MLA) cache.

Four operators, each in a plain form (elementary torch operations, fp32) and through the library:

  keys    tf_block_keys_update        the mean row of every 64-row block that holds new rows
  scores  tf_block_scores             sum_h w_h max(0, scale q_h . k_b) of every visible block b
  blocks  tf_paged_mla_attend_blocks  attention of each query row over its own list of blocks
  shared  tf_paged_mla_attend_shared  attention of streams that share a prefix of pages

A cache row is 512 latent values and 64 rope values; rows lie in 512-row pages (bf16, or E4M3 codes
with one fp32 scale a row, whose latent value is bf16(code * scale)).  Values are N(0, 1), as a
normalised latent has them, so scores of scale 1/sqrt(576) have a deviation of 1.
"""
import math

import torch

own = False

PAGE, LAT, ROPE, DK, BLOCK = 512, 512, 64, 576, 64
PAGE_BYTES = {False: PAGE * DK * 2, True: PAGE * LAT + PAGE * 4 + PAGE * ROPE * 2}
SCALE = DK ** -0.5


def listed():
    return [
        # one decode step of 16 streams: the block that the step's row went to is averaged again
        {"name": "keys_step", "op": "keys", "S": 16, "lo": 30000, "hi": 40960, "new": 1, "fp8": False},
        # the block keys of a whole batch of prompts, after their prefill
        {"name": "keys_batch", "op": "keys", "S": 8, "lo": 4096, "hi": 65536, "new": 0, "fp8": False},
        # the same for one long prompt on FP8 pages
        {"name": "keys_long_fp8", "op": "keys", "S": 1, "lo": 208000, "hi": 208000, "new": 0, "fp8": True},
        # block scores of a decode batch, all heads of a query row choosing together
        {"name": "scores_decode", "op": "scores", "S": 8, "R": 1, "H": 64, "lo": 4096, "hi": 65536, "w": False, "sink": 1, "local": 2},
        # block scores of a prefill chunk of 2,048 rows behind 100,000, with head weights
        {"name": "scores_prefill", "op": "scores", "S": 1, "R": 2048, "H": 64, "lo": 102048, "hi": 102048, "w": True, "sink": 1, "local": 4},
        # one short stream with 16 heads: what a call costs at least
        {"name": "blocks_tiny", "op": "blocks", "S": 1, "R": 1, "H": 16, "lo": 2048, "hi": 2048, "k": 8, "fp8": False},
        # a decode batch of 64 streams, 2,048 rows of each
        {"name": "blocks_decode", "op": "blocks", "S": 64, "R": 1, "H": 64, "lo": 4096, "hi": 32768, "k": 32, "fp8": False},
        # two query rows a stream (a draft and the next token) on FP8 pages, odd lengths
        {"name": "blocks_mtp_fp8", "op": "blocks", "S": 16, "R": 2, "H": 64, "lo": 5001, "hi": 40960, "k": 64, "fp8": True},
        # a prefill chunk: every row attends 2,048 of up to 102,048 rows
        {"name": "blocks_prefill", "op": "blocks", "S": 1, "R": 2048, "H": 64, "lo": 102048, "hi": 102048, "k": 32, "fp8": False},
        # eight answers to one prompt, a few hundred own rows each
        {"name": "shared_batch", "op": "shared", "S": 8, "R": 1, "H": 64, "G": 1, "prefix": 8192, "lo": 1, "hi": 500, "fp8": False},
        # many streams with 16 heads over two system prompts of odd lengths
        {"name": "shared_16_heads", "op": "shared", "S": 64, "R": 1, "H": 16, "G": 2, "prefix": 32767, "lo": 64, "hi": 2000, "fp8": False},
        # draft rows behind a long shared document on FP8 pages
        {"name": "shared_long_fp8", "op": "shared", "S": 8, "R": 2, "H": 64, "G": 1, "prefix": 131072, "lo": 2, "hi": 4096, "fp8": True},
    ]


# ---- sizes that follow from a case -------------------------------------------------------------

def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], the same for every seed."""
    return [lo + int((hi - lo) * ((0.5 + 0.6180339887 * i) % 1.0)) if n > 1 else hi for i in range(n)]


def _prefixes(c):
    """The shared rows of each group: up to a third fewer for the later ones."""
    return [c["prefix"] - g * c["prefix"] // (3 * c["G"]) for g in range(c["G"])]


def _lens(c):
    own_rows = _spread(c["S"], c["lo"], c["hi"])
    if c["op"] != "shared":
        return own_rows
    each = c["S"] // c["G"]
    return [p + n for p, n in zip([p for p in _prefixes(c) for _ in range(each)], own_rows)]


def _blocks_of(n):
    return (n + BLOCK - 1) // BLOCK


def _row_bytes(fp8):
    return LAT + 4 + 2 * ROPE if fp8 else 2 * DK


def work(case):
    c, lens = case, _lens(case)
    if c["op"] == "keys":
        rows = sum(n - (0 if c["new"] == 0 else (n - c["new"]) // BLOCK * BLOCK) for n in lens)
        blocks = sum(_blocks_of(n) - (0 if c["new"] == 0 else (n - c["new"]) // BLOCK) for n in lens)
        return {"bytes": rows * _row_bytes(c["fp8"]) + blocks * 2 * DK, "flops": rows * DK}
    S, R, H = c["S"], c["R"], c["H"]
    pos = [[n - R + r for r in range(R)] for n in lens]
    io = S * R * H * (2 * DK + 2 * LAT + 4)
    if c["op"] == "scores":
        seen = sum(p // BLOCK + 1 for ps in pos for p in ps)
        cols = max(_blocks_of(n) for n in lens)
        read = sum(_blocks_of(n) for n in lens) * 2 * DK + S * R * H * (2 * DK + (4 if c["w"] else 0))
        return {"bytes": read + S * R * cols * 4, "flops": seen * H * (2 * DK + 2)}
    if c["op"] == "blocks":
        # a row attends min(k, visible) blocks, its own one (the last, partly visible) among them
        keys = [sum((min(c["k"], p // BLOCK + 1) - 1) * BLOCK + p % BLOCK + 1 for p in ps) for ps in pos]
        held = [min(n, k) for n, k in zip(lens, keys)]
        return {"bytes": sum(held) * _row_bytes(c["fp8"]) + io + S * R * c["k"] * 4, "flops": 2 * (DK + LAT) * H * sum(keys)}
    each = S // c["G"]
    held = sum(_prefixes(c)) + sum(n - p for n, p in zip(lens, [p for p in _prefixes(c) for _ in range(each)]))
    return {"bytes": held * _row_bytes(c["fp8"]) + io, "flops": 2 * (DK + LAT) * H * sum(p + 1 for ps in pos for p in ps)}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """A case of the listed ones' ranges: from one stream and one row to the largest, odd sizes included."""
    most = {op: max(max(work(c)["bytes"] / 6e3, work(c)["flops"] / 1e6) for c in listed() if c["op"] == op)
            for op in ("keys", "scores", "blocks", "shared")}
    while True:
        op = rng.choice(["keys", "scores", "blocks", "shared"])
        hi = _log(rng, 70, 100000)
        lo = rng.randint(max(1, hi // 16), hi)
        H = rng.choice([1, 5, 8, 16, 20, 32, 64, 96, 128])
        if op == "keys":
            c = {"op": op, "S": _log(rng, 1, 64), "lo": lo, "hi": hi, "new": rng.choice([0, 0, 1, 2, rng.randint(3, 70)]), "fp8": rng.random() < 0.5}
            c["new"] = min(c["new"], lo)
        elif op in ("scores", "blocks"):
            if rng.random() < 0.6:
                S, R = _log(rng, 1, 64), rng.randint(1, 2)
            else:
                S, R = rng.randint(1, 3), _log(rng, 3, 2048)
            c = {"op": op, "S": S, "R": R, "H": H, "lo": max(lo, R), "hi": max(hi, R)}
            if op == "scores":
                c |= {"w": rng.random() < 0.5, "sink": rng.randint(0, 2), "local": rng.randint(1, 5)}
                c["hi"] = max(c["hi"], 2 * (R + BLOCK * (c["sink"] + c["local"] + 1)))   # some block's score decides
            else:
                c |= {"k": _log(rng, 1, 64), "fp8": rng.random() < 0.5}
        else:
            G, R = rng.randint(1, 3), rng.randint(1, 2)
            own_hi = _log(rng, 2, 4096)
            c = {"op": op, "S": G * rng.randint(1, 20), "R": R, "H": H, "G": G, "prefix": _log(rng, 70, 131072), "lo": rng.randint(R, max(R, own_hi // 4)),
                 "hi": max(R, own_hi), "fp8": rng.random() < 0.5}
        w = work(c)
        rows = sum(_lens(c))
        # the plain forms hold each stream's (or row's) keys in fp32: a few GB at most
        held = c["S"] * c["R"] * c["k"] * BLOCK if op == "blocks" else rows
        if max(w["bytes"] / 6e3, w["flops"] / 1e6) <= most[op] and rows <= 2_200_000 and held <= 4_300_000:
            return c


# ---- inputs ------------------------------------------------------------------------------------

def _views(mem, pages, fp8):
    """The pool's blocks as tensors: (latent or codes, scales, rope), one entry a page."""
    off = -mem.data_ptr() % 1024
    raw = mem[off:off + pages * PAGE_BYTES[fp8]].view(pages, PAGE_BYTES[fp8])
    if not fp8:
        x = raw.view(torch.bfloat16)
        return x[:, :PAGE * LAT].unflatten(1, (PAGE, LAT)), None, x[:, PAGE * LAT:].unflatten(1, (PAGE, ROPE))
    a, b = PAGE * LAT, PAGE * LAT + PAGE * 4
    return (raw[:, :a].view(torch.float8_e4m3fn).unflatten(1, (PAGE, LAT)), raw[:, a:b].view(torch.float32),
            raw[:, b:].view(torch.bfloat16).unflatten(1, (PAGE, ROPE)))


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    lens, S, fp8 = _lens(c), c["S"], c.get("fp8", False)
    npg = [(n + PAGE - 1) // PAGE for n in lens]
    shared = [0] * S   # pages that the group's first stream holds for all
    first = list(range(S))
    if c["op"] == "shared":
        each = S // c["G"]
        for s in range(S):
            if s % each:
                shared[s], first[s] = _prefixes(c)[s // each] // PAGE, s - s % each
    pages = sum(npg) - sum(shared) + 2
    ids = torch.randperm(pages, generator=host, dtype=torch.int64).tolist()
    table, at = torch.zeros((S, max(npg)), dtype=torch.int32), 0
    for s in range(S):
        table[s, :shared[s]] = table[first[s], :shared[s]]
        n = npg[s] - shared[s]
        table[s, shared[s]:npg[s]] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    st = {"c": c, "S": S, "fp8": fp8, "lens": lens, "pages": pages, "table": table.to(dev), "max_pages": max(npg),
          "len_t": torch.tensor(lens, device=dev)}
    st["mem"] = mem = torch.empty(pages * PAGE_BYTES[fp8] + 256 + 1024, dtype=torch.uint8, device=dev)
    if c["op"] != "scores":
        lat, scales, rope = _views(mem, pages, fp8)
        if fp8:
            x = torch.randn((pages, PAGE, LAT), generator=g, device=dev)
            scales.copy_(x.abs().amax(-1) / 448)
            lat.copy_((x / scales[..., None]).to(torch.float8_e4m3fn))
            del x
        else:
            lat.normal_(generator=g)
        rope.normal_(generator=g)
        if c["op"] == "shared":
            # the rows of a shared prefix's last, partly shared page are the same in every stream of the group
            each = S // c["G"]
            for s in range(S):
                p = _prefixes(c)[s // each]
                if s % each and p % PAGE:
                    a, b, n = int(table[s - s % each, p // PAGE]), int(table[s, p // PAGE]), p % PAGE
                    for v in (lat.view(torch.uint8) if fp8 else lat, scales, rope):
                        if v is not None:
                            v[b, :n] = v[a, :n]
    if c["op"] == "keys":
        st["bkeys"] = torch.zeros((pages, PAGE // BLOCK, DK), dtype=torch.bfloat16, device=dev)
        st["from"] = [0 if c["new"] == 0 else n - c["new"] for n in lens]
        st["from_t"] = torch.tensor(st["from"], device=dev)
    else:
        R, H = c["R"], c["H"]
        st["q"] = torch.randn((S, R, H, DK), generator=g, device=dev).bfloat16()
        st["pos_t"] = st["len_t"][:, None] - R + torch.arange(R, device=dev)
        st["out"] = torch.empty((S, R, H, LAT), dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.empty((S, R, H), dtype=torch.float32, device=dev)
    if c["op"] == "scores":
        # means of 64 rows of N(0, 1) around a direction of their own
        st["bkeys"] = (torch.randn((pages, PAGE // BLOCK, DK), generator=g, device=dev) * 0.3).bfloat16()
        st["w"] = torch.randn((S, R, H), generator=g, device=dev) if c["w"] else None
        st["cols"] = _blocks_of(max(lens))
        st["scores"] = torch.empty((S * R, (st["cols"] + 3) // 4 * 4), dtype=torch.float32, device=dev)
        st["nblk"] = torch.empty((S * R,), dtype=torch.int32, device=dev)
    elif c["op"] == "blocks":
        # the best blocks of a score that neighbouring rows have in common for the most part, best first
        nb, k = _blocks_of(max(lens)), c["k"]
        x = torch.randn((S, 1, nb), generator=g, device=dev) + 0.5 * torch.randn((S, c["R"], nb), generator=g, device=dev)
        b = torch.arange(nb, device=dev)
        mine = st["pos_t"][..., None] // BLOCK
        x = torch.where((b == 0) & (mine > 0), 1e9, torch.where(b == mine, 2e9, x)).masked_fill(b > mine, -math.inf)
        v, i = torch.topk(x, min(k, nb), -1)
        st["blk"] = torch.full((S, c["R"], k), -1, dtype=torch.int32, device=dev)
        st["blk"][..., :min(k, nb)] = torch.where(v > -math.inf, i, -1).int()
    if own:   # the handle and the workspace that a program keeps
        from paged_mla_kv_gb300 import binding as B
        st["pool"] = B.KVPool(1, pages, memory=mem, fp8=fp8)
        n = 0
        if c["op"] == "blocks":
            n = B.tf_paged_mla_blocks_workspace_bytes(st["pool"], S, c["R"], c["H"], lens, c["k"])
        elif c["op"] == "shared":
            n = B.tf_paged_mla_shared_workspace_bytes(st["pool"], S, c["R"], c["H"], lens, [S // c["G"]] * c["G"], _prefixes(c))
        st["ws"] = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    return st


# ---- one pass ----------------------------------------------------------------------------------

def run(st):
    c = st["c"]
    if own:
        return _library(st, c)
    return {"keys": _keys, "scores": _scores, "blocks": _blocks, "shared": _shared}[c["op"]](st, c)


def _library(st, c):
    from paged_mla_kv_gb300 import binding as B
    pool, pt, mp, lens = st["pool"], st["table"], st["max_pages"], st["lens"]
    if c["op"] == "keys":
        B.tf_block_keys_update(pool, 0, pt, mp, st["from"], lens, st["bkeys"])
        return st["bkeys"]
    if c["op"] == "scores":
        B.tf_block_scores(pool, st["bkeys"], pt, mp, lens, st["q"], SCALE, st["scores"], w=st["w"], nblk=st["nblk"], sink=c["sink"], local=c["local"])
        return {"scores": st["scores"][:, :st["cols"]], "nblk": st["nblk"]}
    if c["op"] == "blocks":
        B.tf_paged_mla_attend_blocks(pool, 0, pt, mp, lens, st["blk"], st["q"], SCALE, st["out"], st["lse"], st["ws"])
    else:
        G = c["G"]
        B.tf_paged_mla_attend_shared(pool, 0, pt, mp, lens, [c["S"] // G] * G, _prefixes(c), st["q"], SCALE, st["out"], st["lse"], st["ws"])
    return {"out": st["out"], "lse": st["lse"]}


def _rows(st, page, row):
    """Cache rows in fp32, 576 wide, at (page, row) index tensors of one shape."""
    lat, scales, rope = _views(st["mem"], st["pages"], st["fp8"])
    if st["fp8"]:
        x = (lat.view(torch.uint8)[page, row].view(torch.float8_e4m3fn).float() * scales[page, row][..., None]).bfloat16()
    else:
        x = lat[page, row]
    return torch.cat([x, rope[page, row]], -1).float()


def _keys(st, c):
    nb, b0 = (st["len_t"] + BLOCK - 1) // BLOCK, st["from_t"] // BLOCK
    count = nb - b0
    total = sum(_blocks_of(n) - f // BLOCK for n, f in zip(st["lens"], st["from"]))
    s = torch.repeat_interleave(torch.arange(st["S"], device=count.device), count, output_size=total)
    b = torch.arange(total, device=count.device) - (count.cumsum(0) - count)[s] + b0[s]
    page = st["table"][s, b // 8].long()
    i = torch.arange(BLOCK, device=count.device)
    x = _rows(st, page[:, None].expand(-1, BLOCK), (b % 8 * BLOCK)[:, None] + i)
    there = b[:, None] * BLOCK + i < st["len_t"][s][:, None]
    mean = torch.where(there[..., None], x, 0.0).sum(1) / there.sum(1, keepdim=True)
    st["bkeys"][page, b % 8] = mean.bfloat16()
    return st["bkeys"]


def _scores(st, c):
    b = torch.arange(st["cols"], device="cuda")
    k = st["bkeys"][st["table"].long()].flatten(1, 2)[:, :st["cols"]].float()   # [S][blocks][576]
    dots = SCALE * torch.einsum("srhd,sbd->srhb", st["q"].float(), k)
    x = dots.clamp_min(0)
    x = (x if st["w"] is None else x * st["w"][..., None]).sum(2)
    mine = st["pos_t"][..., None] // BLOCK
    x = torch.where((b < c["sink"]) | (b > mine - c["local"]), math.inf, x)
    x = torch.where(b <= mine, x, -math.inf)
    return {"scores": x.flatten(0, 1), "nblk": (mine + 1).int().flatten()}


def _softmax_av(s, seen, v):
    """(out in bf16, lse) of scores s [.., H, n], a mask that broadcasts to them and values [.., n, 512]."""
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m > -math.inf, m, 0.0))
    total = e.sum(-1, keepdim=True)
    out = torch.where(total > 0, torch.matmul(e, v) / total, 0.0)
    return {"out": out.bfloat16(), "lse": (m + torch.log(total))[..., 0]}


def _blocks(st, c):
    blk = st["blk"].long()
    i = (blk.clamp_min(0)[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten(2)   # [S][R][k * 64]
    seen = (blk >= 0).repeat_interleave(BLOCK, -1) & (i <= st["pos_t"][..., None])
    i = torch.minimum(i, st["len_t"][:, None, None] - 1)
    page = torch.gather(st["table"].long()[:, None].expand(-1, c["R"], -1), 2, i // PAGE)
    x = _rows(st, page, i % PAGE)
    return _softmax_av(SCALE * torch.matmul(st["q"].float(), x.transpose(-1, -2)), seen[:, :, None], x[..., :LAT])


def _shared(st, c):
    n = max(st["lens"])
    i = torch.arange(n, device="cuda")
    x = _rows(st, st["table"].long()[:, i // PAGE], (i % PAGE).expand(st["S"], -1))   # [S][n][576]
    q = st["q"].float().flatten(1, 2)
    seen = (i <= st["pos_t"][..., None]).repeat_interleave(c["H"], 1)
    o = _softmax_av(SCALE * torch.matmul(q, x.transpose(1, 2)), seen, x[..., :LAT])
    return {"out": o["out"].view_as(st["out"]), "lse": o["lse"].view_as(st["lse"])}


# ---- the definitions in 64 bits ----------------------------------------------------------------

def _stream64(st, s):
    """Stream s's rows one after another, in fp64."""
    n = st["lens"][s]
    ids = st["table"][s, :(n + PAGE - 1) // PAGE].long()
    lat, scales, rope = _views(st["mem"], st["pages"], st["fp8"])
    if st["fp8"]:
        lat = torch.stack([lat[p].float() * scales[p][:, None] for p in ids.tolist()]).to(torch.bfloat16)
    else:
        lat = lat[ids]
    return torch.cat([lat.double(), rope[ids].double()], 2).view(-1, DK)[:n]


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    c, lens = case, st["lens"]
    if c["op"] == "keys":
        res = st["bkeys"].double()
        for s, n in enumerate(lens):
            x, b0 = _stream64(st, s), st["from"][s] // BLOCK
            whole = n // BLOCK
            means = list(x[:whole * BLOCK].view(whole, BLOCK, DK).mean(1)[b0:]) if whole > b0 else []
            if n % BLOCK:
                means.append(x[whole * BLOCK:].mean(0))
            t = st["table"][s].tolist()
            at = torch.tensor([t[b // 8] * 8 + b % 8 for b in range(b0, b0 + len(means))], device="cuda")
            res.view(-1, DK)[at] = torch.stack(means)
        return res
    q, R, H = st["q"].double(), c["R"], c["H"]
    if c["op"] == "scores":
        res = torch.full((c["S"] * R, st["cols"]), -math.inf, dtype=torch.float64, device="cuda")
        for s, n in enumerate(lens):
            nb = _blocks_of(n)
            k = st["bkeys"][st["table"][s, :(nb + 7) // 8].long()].double().reshape(-1, DK)[:nb]
            for a in range(0, R, 256):
                x = torch.relu(q[s, a:a + 256].reshape(-1, DK) @ k.T * SCALE).view(-1, H, nb)
                x = x.sum(1) if st["w"] is None else torch.bmm(st["w"][s, a:a + 256, None].double(), x)[:, 0]
                for r in range(x.shape[0]):
                    mine = (n - R + a + r) // BLOCK
                    line = res[s * R + a + r]
                    line[:mine + 1] = x[r, :mine + 1]
                    line[:min(c["sink"], mine + 1)] = math.inf
                    line[max(0, mine - c["local"] + 1):mine + 1] = math.inf
        return {"scores": res, "nblk": None}
    out = torch.zeros((c["S"], R, H, LAT), dtype=torch.float64, device="cuda")
    lse = torch.full((c["S"], R, H), -math.inf, dtype=torch.float64, device="cuda")
    for s, n in enumerate(lens):
        x = _stream64(st, s)
        lists = st["blk"][s].cpu().tolist() if c["op"] == "blocks" else None
        for r in range(R):
            p = n - R + r
            if lists is None:
                keys = x[:p + 1]
            else:
                keys = torch.cat([x[b * BLOCK:min(b * BLOCK + BLOCK, p + 1)] for b in lists[r] if b >= 0])
            t = q[s, r] @ keys.T * SCALE
            lse[s, r] = torch.logsumexp(t, 1)
            out[s, r] = torch.softmax(t, 1) @ keys[:, :LAT]
    return {"out": out, "lse": lse}
