"""Serving from an 8-bit paged KV cache with rotary positions: the operators'
cases, their plain forms in elementary torch operations, and the calls a user
makes.

A step of a model whose positions are rotations: the queries are rotated
(``attn_rotary``); the new K and V rows go into the paged cache, K rotated on the
way, in 16 bits (``attn_cache_append_rotary``) or in 8 (``attn_qcache_append``,
with a scale for each page and KV head); over the 8-bit cache each sequence's
last tokens attend to everything up to themselves (``attn_qcache_attend``).

The operators (float sums in 32 bits or more, each output rounded once):

  rotary   pairs of the first `rot` values of a head, (x[i], x[i + rot/2]) or,
           interleaved, (x[2i], x[2i+1]), are turned by the angle a = p w[i] at
           position p: (x cos a - y sin a, x sin a + y cos a) m.
           w[i] = f (g + (1 - g) / stretch), f = base^(-2i/rot),
           g = clamp((t - low) / (high - low), 0, 1), t = original f / 2 pi
           (positions that turn often keep their rate, those that turn seldom
           are slowed by `stretch`); m is a factor of the whole
  append   every kept row goes to its sequence's next position, K turned by that
           position, new pages being the lowest ones that nobody holds
  append8  the same into e4m3 codes: per layer, page and head, of K and of V, the
           scale is s = 2^e, e the least whole number from -100 on with
           |x| <= 448 * 2^e for every row the page has taken since its first;
           a value's code is x / s rounded to the nearest e4m3 (ties to even).
           Where s grows the page's earlier codes are rounded anew to it.
  attend   o[i,h] = sum_l softmax_l(q[i,h] . K[l] / sqrt(D)) V[l], K and V codes
           times their page's and head's scale, l up to row i's own position
           len - n + i of a sequence with n rows
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
F8 = torch.float8_e4m3fn


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one token's queries, a quarter of each head rotated, cut out of a fused projection's row
        dict(name="rotary-token", op="rotary", n=1, heads=16, D=256, rot=64, inter=False, long=False, top=5000,
             wide=1024, dtype="bf16"),
        # a long prompt's queries, the whole head in interleaved pairs, positions stretched far beyond training
        dict(name="rotary-prompt", op="rotary", n=8191, heads=16, D=256, rot=256, inter=True, long=True, top=1000000,
             wide=0, dtype="bf16"),
        # one new token for each chat of a batch, after the last step's rejected tokens are cut off
        dict(name="append-step", op="append", B=24, n=1, layers=10, Hkv=2, D=256, page=64, len=5000, rot=64,
             inter=False, long=False, dtype="bf16"),
        # a chunk of every prompt of a batch
        dict(name="append-chunk", op="append", B=24, n=500, layers=10, Hkv=2, D=256, page=64, len=2100, rot=256,
             inter=True, long=True, dtype="bf16"),
        # the 8-bit cache: one new token for each chat of a batch (some pages' scales grow)
        dict(name="append8-step", op="append8", B=48, n=1, layers=10, Hkv=2, D=256, page=64, len=5000, rot=64,
             inter=False, long=False, dtype="bf16"),
        # a chunk of every prompt into the 8-bit cache, fp16 rows, larger pages
        dict(name="append8-chunk", op="append8", B=24, n=500, layers=10, Hkv=2, D=256, page=128, len=2100, rot=256,
             inter=False, long=True, dtype="fp16"),
        # a chat's next token over a short cache
        dict(name="attend-single", op="attend", B=1, n=1, Hq=16, Hkv=2, D=256, page=64, len=700, ragged=0,
             dtype="bf16"),
        # a server's batch, one token each, caches of uneven length
        dict(name="attend-batch", op="attend", B=48, n=1, Hq=16, Hkv=2, D=256, page=64, len=9001, ragged=3,
             dtype="bf16"),
        # the few drafted tokens of one chat over a long context
        dict(name="attend-long", op="attend", B=1, n=5, Hq=16, Hkv=2, D=256, page=128, len=131000, ragged=0,
             dtype="bf16"),
        # smaller heads in fp16, small pages, many KV heads
        dict(name="attend-heads", op="attend", B=64, n=2, Hq=32, Hkv=8, D=128, page=16, len=3001, ragged=5,
             dtype="fp16"),
        # a chunk of a few prompts over what is cached of them
        dict(name="attend-chunk", op="attend", B=4, n=500, Hq=16, Hkv=2, D=256, page=64, len=8000, ragged=1,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    tops = {}
    for c in listed():
        w = work(c)
        t = tops.setdefault(c["op"], [0.0, 0.0])
        t[0], t[1] = max(t[0], w["bytes"]), max(t[1], w["flops"])
    op = rng.choice(["rotary", "append", "append8", "append8", "attend", "attend", "attend"])
    while True:
        D = rng.choice([64, 128, 256, 256])
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        turn = dict(rot=rng.choice([r for r in (16, 32, 48, 64, 128, 256) if r <= D]), inter=rng.random() < 0.5,
                    long=rng.random() < 0.4)
        if op == "rotary":
            c = dict(op=op, n=_log(rng, 1, 16384), heads=_log(rng, 1, 64), D=D, top=_log(rng, 1000, 1000000),
                     wide=rng.choice([0, 0, 8, 1000]), dtype=dtype, **turn)
        elif op != "attend":
            c = dict(op=op, B=_log(rng, 1, 64), n=_log(rng, 1, 500), layers=rng.choice([1, 4, 10]),
                     Hkv=rng.choice([1, 2, 3, 8]), D=D, page=rng.choice([16, 32, 64, 128, 256]), len=_log(rng, 1, 5000),
                     dtype=dtype, **turn)
            if _pool_rows(c) * c["layers"] * c["Hkv"] * c["D"] > 48 * 5200 * 10 * 512:
                continue
        else:
            Hkv = rng.choice([1, 2, 4, 8])
            c = dict(op=op, B=_log(rng, 1, 96), n=_log(rng, 1, 500) if rng.random() < 0.4 else rng.randint(1, 5),
                     Hq=Hkv * rng.choice([1, 2, 4, 5, 8, 16]), Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128, 256]),
                     len=_log(rng, 1, 131000), ragged=rng.randrange(6), dtype=dtype)
            pairs = c["B"] * c["n"] * c["len"] * c["Hq"]
            if c["B"] * c["len"] * Hkv * D > 64 * 3001 * 1024 or pairs > 4 * 500 * 8000 * 16 or c["Hq"] > 64:
                continue
        w = work(c)
        if w["bytes"] <= tops[op][0] and w["flops"] <= tops[op][1]:
            return c


# ---------------------------------------------------- shapes that a case fixes

def _lens(c):
    """Cached tokens per sequence."""
    if c["op"] == "attend":
        if not c["ragged"]:
            return [max(c["len"], c["n"])] * c["B"]
        r = random.Random(c["ragged"])
        return [max(1, c["n"], int(c["len"] * (1.0 if b == 0 else 0.125 + 0.875 * r.random()))) for b in range(c["B"])]
    return [max(1, c["len"] - 13 * b % max(1, c["len"] // 2)) for b in range(c["B"])]


def _counts(c):
    """Rows per sequence: up to n, uneven."""
    if c["op"] == "attend":
        return [max(1, c["n"] - b % 3) if c["ragged"] else c["n"] for b in range(c["B"])]
    return [max(1, c["n"] - (37 * b) % (c["n"] // 2 + 1)) for b in range(c["B"])]


def _cut(L):
    """Tokens that stay when the last step's are taken back."""
    return max(0, L - 3)


def _pages(rows, page):
    return -(-rows // page)


def _pool_rows(c):
    """Rows of the page pool of a case (a quarter of its pages stays free)."""
    need = c["B"] * _pages(max(c["len"], c["n"]) + (0 if c["op"] == "attend" else c["n"]), c["page"])
    return (need + need // 4 + 8) * c["page"]


def work(case):
    c = case
    if c["op"] == "rotary":
        values = c["n"] * c["heads"] * c["D"]
        return {"bytes": 4.0 * values + 4.0 * c["n"], "flops": 3.0 * c["n"] * c["heads"] * c["rot"]}
    if c["op"] == "attend":
        lens, counts = _lens(c), _counts(c)
        seen = sum(n * L - n * (n - 1) // 2 for L, n in zip(lens, counts))
        scales = sum(_pages(L, c["page"]) for L in lens) * c["Hkv"] * 8
        return {"bytes": float(2 * sum(lens) * c["Hkv"] * c["D"] + scales + 4 * sum(counts) * c["Hq"] * c["D"]),
                "flops": 4.0 * seen * c["Hq"] * c["D"]}
    rows = sum(_counts(c))
    values = rows * c["layers"] * c["Hkv"] * c["D"]  # of K, and of V
    return {"bytes": float(values * 2 * (4 if c["op"] == "append" else 3)),
            "flops": 3.0 * rows * c["layers"] * c["Hkv"] * c["rot"]}


# -------------------------------------------------------------------- inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _offsets(counts):
    return _ints(np.concatenate([[0], np.cumsum(counts)]).tolist())


#: stretch, low, high, original length, factor: none, and 32 times the length that a model was trained on
PLAIN, LONG = (1.0, 0.0, 0.0, 0, 1.0), (32.0, 1.0, 32.0, 8192, 1.25)
BASE = 1000000.0


def _rates(c):
    """Radians a position for each pair, and the factor of the whole."""
    stretch, low, high, original, factor = LONG if c["long"] else PLAIN
    f = BASE ** (-np.arange(0, c["rot"], 2, dtype=np.float64) / c["rot"])
    if stretch != 1.0:
        g = np.clip((original * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
        f = f * (g + (1.0 - g) / stretch)
    return f, factor


def _tables(c, g, lens, spare):
    """Page tables: the sequences hold `lens` tokens in pages scattered over the pool."""
    page, P = c["page"], _pool_rows(c) // c["page"]
    order = torch.randperm(P, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    width = max(_pages(L + spare, page) for L in lens)
    used = [_pages(L, page) for L in lens]
    start = np.concatenate([[0], np.cumsum(used)])
    j = torch.arange(width, device=DEV)[None]
    u, s0 = _ints(used)[:, None], _ints(start[:-1].tolist())[:, None]
    table = torch.where(j < u, order[(s0 + j).clamp(max=P - 1).long()], -1).contiguous()
    refs = torch.zeros(P, dtype=torch.int32, device=DEV)
    refs[order[:int(start[-1])].long()] = 1
    return dict(refs=refs, table=table, lens=_ints(lens), status=torch.zeros(4, dtype=torch.int32, device=DEV))


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * seed + 29)
    s = {"case": c}

    def normal(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=g)

    def pool8(layers):
        """Codes and scales as appends leave them: heads of different size, most pages full of one scale's values."""
        P = _pool_rows(c) // c["page"]
        codes = normal(layers, P, c["page"], c["Hkv"], c["D"], dtype=torch.bfloat16).mul_(90.0).clamp_(-448, 448).to(F8)
        e = torch.randint(-9, -4, (1, 1, c["Hkv"]), generator=g, device=DEV) + \
            torch.randint(0, 2, (layers, P, c["Hkv"]), generator=g, device=DEV)
        return codes, torch.exp2(e.float())

    if "rot" in c:
        s["rates"] = torch.from_numpy(_rates(c)[0]).to(DEV)
    if c["op"] == "rotary":
        row = c["heads"] * c["D"]
        s["x"] = normal(c["n"], row + c["wide"], dtype=TYPES[c["dtype"]])[:, :row].unflatten(1, (c["heads"], c["D"]))
        s["positions"] = torch.randint(0, c["top"], (c["n"],), generator=g, device=DEV, dtype=torch.int32)
        s["o"] = torch.zeros(c["n"], c["heads"], c["D"], dtype=TYPES[c["dtype"]], device=DEV)
    else:
        lens, counts, t = _lens(c), _counts(c), TYPES[c["dtype"]]
        N = sum(counts)
        s["offsets"] = _offsets(counts)
        s["cache"] = _tables(c, g, lens, 0 if c["op"] == "attend" else c["n"])
        layers = c.get("layers", 1)
        if c["op"] == "append":
            shape = (layers, _pool_rows(c) // c["page"], c["page"], c["Hkv"], c["D"])
            s["cache"] |= {n: normal(*shape, dtype=t) for n in ("k", "v")}
        else:
            for n in ("k", "v"):
                s["cache"][n], s["cache"][n + "_scale"] = pool8(layers)
        if c["op"] == "attend":
            s["q"] = normal(N, c["Hq"], c["D"], dtype=t)
            s["o"] = torch.zeros_like(s["q"])
        else:
            # what the step before left behind: some of the cached tokens are taken back first
            s["cut"] = _ints([_cut(L) for L in lens])
            size = torch.exp2(torch.randint(-2, 2, (1, 1, c["Hkv"], 1), generator=g, device=DEV).float())
            for n in ("k_new", "v_new"):
                s[n] = (normal(layers, N, c["Hkv"], c["D"], dtype=t) * size.to(t)).contiguous()
    if own:
        _handles(s)
    return s


def _handles(s):
    """The handles and the workspace that a user's program keeps."""
    import bit_grouped_expert_gb300 as moe
    c, need = s["case"], 0
    if "rot" in c:
        stretch, low, high, original, factor = LONG if c["long"] else PLAIN
        s["turn"] = moe.make_rotary(c["rot"], base=BASE, interleaved=c["inter"], stretch=stretch, low_turns=low,
                                    high_turns=high, original_len=original, factor=factor)
    if "cache" in s:
        k = s["cache"]
        tables = (k["refs"], k["table"], k["lens"], k["status"])
        if c["op"] == "append":
            s["handle"] = moe.make_attn_cache(k["k"], k["v"], *tables)
            need = moe.attn_cache_append_workspace_bytes(s["handle"], c["B"], s["k_new"].shape[1])
        else:
            s["handle"] = moe.make_attn_qcache(k["k"], k["v"], k["k_scale"], k["v_scale"], *tables)
            if c["op"] == "append8":
                need = moe.attn_qcache_append_workspace_bytes(s["handle"], c["B"], s["k_new"].shape[1])
            else:
                need = moe.attn_qcache_attend_workspace_bytes(s["handle"], c["B"], s["q"].shape[0], c["n"], c["Hq"])
    s["ws"] = torch.zeros(max(need, 16), dtype=torch.uint8, device=DEV)


# ----------------------------------------------------------------- the passes

def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    return {"rotary": _rotary, "append": _append, "append8": _append, "attend": _attend}[c["op"]](s, c)


def _run_own(s, c):
    import bit_grouped_expert_gb300 as moe
    if c["op"] == "rotary":
        moe.attn_rotary(s["turn"], s["x"], s["positions"], s["o"])
        return {"o": s["o"]}
    if c["op"] == "attend":
        moe.attn_qcache_attend(s["handle"], 0, s["q"], s["offsets"], c["B"], c["n"], s["ws"], s["o"])
        return {"o": s["o"]}
    if c["op"] == "append":
        moe.attn_cache_trim(s["handle"], None, s["cut"], c["B"])
        moe.attn_cache_append_rotary(s["handle"], s["turn"], s["k_new"], s["v_new"], s["offsets"], c["B"], s["ws"])
    else:
        moe.attn_qcache_trim(s["handle"], None, s["cut"], c["B"])
        moe.attn_qcache_append(s["handle"], s["turn"], s["k_new"], s["v_new"], s["offsets"], c["B"], s["ws"])
    return _cache_out(s)


def _cache_out(s):
    # (8-bit pools are e4m3 tensors: their values are the codes', to be taken times the scales)
    return {n: s["cache"][n] for n in ("k", "v", "k_scale", "v_scale", "refs", "table", "lens") if n in s["cache"]}


def _turned(x, positions, s, c):
    """x [.., rows, heads, D] in 32 bits, rotated by the rows' positions (angles in 64 bits)."""
    rot, factor = c["rot"], _rates(c)[1]
    a = positions.double()[:, None, None] * s["rates"]
    cos, sin = torch.cos(a).float() * factor, torch.sin(a).float() * factor
    if c["inter"]:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)
    else:
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([u * cos - v * sin, u * sin + v * cos], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _rotary(s, c):
    return {"o": _turned(s["x"].float(), s["positions"], s, c).to(s["x"].dtype)}


def _append(s, c):
    cache, page, B = s["cache"], c["page"], c["B"]
    table, refs = cache["table"], cache["refs"]
    # the cut: pages wholly behind the new length are given up
    j = torch.arange(table.shape[1], device=DEV)[None]
    gone = (j >= ((s["cut"] + page - 1) // page)[:, None]) & (table >= 0)
    refs.index_add_(0, table.clamp(min=0).reshape(-1), -gone.reshape(-1).to(torch.int32))
    table.copy_(torch.where(gone, -1, table))
    cache["lens"].copy_(s["cut"])
    # the new pages
    old, off = cache["lens"].clone(), s["offsets"]
    keep = off[1:] - off[:-1]
    have, want = (old + page - 1) // page, (old + keep + page - 1) // page
    need = want - have
    first = need.cumsum(0) - need
    free = torch.sort((refs != 0).to(torch.uint8), stable=True).indices.to(torch.int32)
    new = (j >= have[:, None]) & (j < want[:, None])
    pages = free[(first[:, None] + j - have[:, None]).clamp(min=0, max=free.numel() - 1).long()]
    table.copy_(torch.where(new, pages, table))
    refs.index_add_(0, torch.where(new, pages, 0).reshape(-1), new.reshape(-1).to(torch.int32))
    cache["lens"].add_(keep)
    # every row's place
    row = torch.arange(s["k_new"].shape[1], device=DEV)
    b = torch.searchsorted(off[1:], row.to(torch.int32), right=True)
    pos = old[b] + row.to(torch.int32) - off[b]
    at = table[b, (pos // page).long()].long()
    k = _turned(s["k_new"].float(), pos, s, c)
    if c["op"] == "append":
        for pool, rows in ((cache["k"], k), (cache["v"], s["v_new"])):
            pool.view(c["layers"], -1, c["Hkv"], c["D"])[:, at * page + pos % page] = rows.to(pool.dtype)
        return _cache_out(s)
    kept = torch.where((old % page > 0) & (keep > 0), table.gather(1, (old // page).clamp(max=table.shape[1] - 1)
                                                                   .long()[:, None])[:, 0], -1)  # pages that go on
    _quantise(cache["k"], cache["k_scale"], k, at, pos, kept, old, c)
    _quantise(cache["v"], cache["v_scale"], s["v_new"].float(), at, pos, kept, old, c)
    return _cache_out(s)


def _quantise(pool, scales, x, at, pos, kept, old, c):
    page = c["page"]
    most = torch.zeros_like(scales).index_reduce_(1, at, x.abs().amax(-1), "amax")
    m, e = torch.frexp(most.double() / 448.0)
    fresh = torch.exp2(torch.where(m > 0.5, e, e - 1).clamp(min=-100).where(most > 0, -100).float())
    touched = torch.zeros(scales.shape[1], dtype=torch.bool, device=DEV).index_fill_(0, at, True)
    on = torch.zeros(scales.shape[1] + 1, dtype=torch.bool, device=DEV)
    on[kept.long()] = True                                # (-1: the last, of no page)
    on = on[:-1]
    to = torch.where((touched & ~on)[None, :, None], fresh, torch.where(touched[None, :, None], fresh.maximum(scales),
                                                                        scales))
    # earlier rows of the pages that go on, to the new scale
    p = kept.clamp(min=0).long()
    codes = pool.view(torch.uint8)
    was = codes[:, p]                                     # [layers, B, page, heads, D]
    f = (scales / to)[:, p][:, :, None, :, None]
    again = (was.view(F8).float() * f).to(F8).view(torch.uint8)
    mine = (torch.arange(page, device=DEV)[None] < (old % page)[:, None]) & (kept >= 0)[:, None]
    rows = (p[:, None] * page + torch.arange(page, device=DEV))[mine]
    flat = codes.view(c["layers"], -1, c["Hkv"], c["D"])
    flat[:, rows] = again[:, mine]
    scales.copy_(to)
    flat[:, at * page + pos % page] = (x / to[:, at][..., None]).to(F8).view(torch.uint8)


def _attend(s, c):
    cache, n, Hkv, G, D, B = s["cache"], c["n"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"], c["B"]
    off = s["offsets"].long()
    i = torch.arange(n, device=DEV)
    count = off[1:] - off[:-1]
    real = i[None] < count[:, None]                                                  # [B, n]
    rows = (off[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    table = cache["table"].long().clamp(min=0)
    L = table.shape[1] * c["page"]
    k, v = ((cache[x].view(torch.uint8)[0][table].view(F8).float() * cache[x + "_scale"][0][table][:, :, None, :, None])
            .reshape(B, L, Hkv, D) for x in ("k", "v"))
    last = cache["lens"][:, None] - count[:, None] + i                               # a row's own position
    mask = (torch.arange(L, device=DEV) <= last[:, :, None]) & real[:, :, None]      # [B, n, L]
    v = torch.where(mask.any(1)[:, :, None, None], v, 0.0)
    q = s["q"][rows].float().reshape(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    a = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(D ** -0.5).reshape(B, Hkv, G, n, L)
    a = a.masked_fill_(~mask[:, None, None], float("-inf"))
    a = torch.exp(a - a.amax(-1, keepdim=True).clamp(min=-3e38))
    den = a.sum(-1, keepdim=True)
    o = torch.matmul(a.reshape(B, Hkv, G * n, L), v.permute(0, 2, 1, 3)).reshape(B, Hkv, G, n, D)
    o = torch.where(den > 0, o / den, 0.0).permute(0, 3, 1, 2, 4).reshape(B, n, c["Hq"], D)
    return {"o": o[real].to(s["q"].dtype)}


# ------------------------------------------------------- values in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"rotary": _exact_rotary, "append": _exact_pages, "append8": _exact_pages,
            "attend": _exact_attend}[case["op"]](s, case)


def _exact_turn(x, positions, c):
    """Complex numbers times e^(i p w): x [.., rows, heads, D] in 64 bits."""
    w, factor = _rates(c)
    z = torch.polar(torch.full((1,), factor, dtype=torch.float64, device=DEV),
                    torch.outer(positions.double(), torch.tensor(w, device=DEV)))[:, None]
    y, h = x.clone(), c["rot"] // 2
    first, second = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["inter"] else (slice(0, h), slice(h, 2 * h))
    t = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * z
    y[..., first], y[..., second] = t.real, t.imag
    return y


def _exact_rotary(s, c):
    return {"o": _exact_turn(s["x"].double(), s["positions"], c)}


def _exact_pages(s, c):
    cache, page, shape = s["cache"], c["page"], (c["layers"], -1, c["Hkv"], c["D"])
    refs, table, lens = (cache[n].cpu().numpy().copy() for n in ("refs", "table", "lens"))
    for b, new in enumerate(s["cut"].tolist()):
        for j in range(_pages(new, page), table.shape[1]):
            if table[b, j] >= 0:
                refs[table[b, j]] -= 1
                table[b, j] = -1
        lens[b] = new
    free = iter(np.flatnonzero(refs == 0).tolist())
    off, parts = s["offsets"].tolist(), []                # parts: (page, its first new row, rows, where they begin)
    where = np.zeros(off[-1], np.int64)
    for b in range(c["B"]):
        for r in range(off[b], off[b + 1]):
            if lens[b] % page == 0:
                table[b, lens[b] // page] = got = next(free)
                refs[got] = 1
            if lens[b] % page == 0 or r == off[b]:
                parts.append([int(table[b, lens[b] // page]), r, 0, int(lens[b]) % page])
            parts[-1][2] += 1
            where[r] = lens[b]
            lens[b] += 1
    tables = {"refs": torch.from_numpy(refs), "table": torch.from_numpy(table), "lens": torch.from_numpy(lens)}
    if len(parts) > 2000:
        return None
    k = _exact_turn(s["k_new"].double(), torch.from_numpy(where).to(DEV), c)
    out = {}
    for name, rows in (("k", k), ("v", s["v_new"].double())):
        pool = cache[name].double()
        if c["op"] == "append":
            for p, r, n, i in parts:
                pool[:, p, i:i + n] = rows[:, r:r + n]
        else:
            scale = cache[name + "_scale"].double()
            for p, r, n, i in parts:
                x = rows[:, r:r + n]
                most = x.abs().amax((1, 3)).clamp(min=448.0 * 2.0 ** -100)
                new = torch.exp2(torch.round(torch.log2(most / 448.0)) - 1)    # at most one power of two too low, or two
                new = torch.where(most > 448.0 * new, 2 * new, new)
                new = torch.where(most > 448.0 * new, 2 * new, new)
                if i:
                    new = torch.maximum(new, scale[:, p])
                    pool[:, p, :i] = _nearest(pool[:, p, :i] * (scale[:, p] / new)[:, None, :, None])
                scale[:, p] = new
                pool[:, p, i:i + n] = _nearest(x / new[:, None, :, None])
            out[name + "_scale"] = scale
        out[name] = pool
    return {**out, **tables}


def _nearest(x):
    """The nearest e4m3 value, ties to even: steps of an eighth of the value's power of two, 2^-9 at least."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_attend(s, c):
    if work(c)["flops"] > 3e11:
        return None
    off, lens, page, G = s["offsets"].tolist(), s["cache"]["lens"].tolist(), c["page"], c["Hq"] // c["Hkv"]
    out = []
    for b in range(c["B"]):
        lo, hi, L = off[b], off[b + 1], lens[b]
        pages = s["cache"]["table"][b].long()[:_pages(L, page)]
        k, v = ((s["cache"][n][0].float()[pages].double() * s["cache"][n + "_scale"][0][pages].double()[:, None, :, None])
                .reshape(-1, c["Hkv"], c["D"])[:L] for n in ("k", "v"))
        hidden = torch.arange(L, device=DEV)[None] > torch.arange(L - (hi - lo), L, device=DEV)[:, None]
        o = torch.empty(hi - lo, c["Hq"], c["D"], dtype=torch.float64, device=DEV)
        for h in range(c["Hq"]):
            a = (s["q"][lo:hi, h].double() @ k[:, h // G].T) / math.sqrt(c["D"])
            o[:, h] = torch.softmax(a.masked_fill(hidden, -np.inf), -1) @ v[:, h // G]
        out.append(o)
    return {"o": torch.cat(out)}
