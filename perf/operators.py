"""Speculative decoding over a paged KV cache: the operators' cases, their plain
forms in elementary torch operations, and the calls a user makes.

A decoding step of a sequence with drafted tokens: every attention layer runs
``attn_tree`` (the tree of drafted tokens against the sequence's cache pages and
their own ancestors), ``moe_draft_verify`` walks the tree with the target's
probabilities and given random numbers, and ``attn_cache_append`` stores the K
and V rows of the accepted path, of all layers, behind the cache.
``attn_cache_fork`` and ``attn_cache_trim`` share, copy, cut and free pages.

The operators (float sums in 32 bits or more, each output rounded once):

  tree    o[i,h] = sum_l softmax_l(s)[l] v[l], s[l] = scale q[i,h] . k[l], over the
          cached positions of the node's sequence, the node and its ancestors;
          parent[i] < i within the tree, -1 a root, -2 padding (output 0)
  verify  from node 0, children in index order: child j (token x) of the current
          node c is taken if u[j] S q_c(x) < R(x), where at first R = p_c, S = 1;
          a child not taken leaves R <- max(R - S q_c, 0), S <- sum R (without q:
          R(x) <- 0, S <- S - R(x)).  At the end the next token is the lowest t
          with R(0) + .. + R(t) > u' sum R.
  append  every kept row goes to its sequence's next position, new pages being
          the lowest ones that nobody holds
  fork    full pages are shared (one more holder), the last, partly filled page is
          copied to the lowest free page
  trim    pages wholly behind the new length lose a holder, their table entries
          become -1
"""
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # a chat's next token with nothing drafted: one token over a short cache
        dict(name="tree-single", op="tree", B=1, n=1, shape="chain", Hq=16, Hkv=2, D=256, page=64, len=700, ragged=0,
             dtype="bf16"),
        # a server's batch with four drafted tokens each, caches of uneven length
        dict(name="tree-batch", op="tree", B=24, n=5, shape="chain", Hq=16, Hkv=2, D=256, page=64, len=9001, ragged=3,
             dtype="bf16"),
        # a wide draft tree over one long context
        dict(name="tree-long", op="tree", B=1, n=61, shape="tree", Hq=16, Hkv=2, D=256, page=128, len=131000,
             ragged=0, dtype="bf16"),
        # smaller heads in fp16, small pages, a tree on each of many short caches
        dict(name="tree-fp16", op="tree", B=48, n=16, shape="tree", Hq=32, Hkv=8, D=128, page=16, len=3001, ragged=5,
             dtype="fp16"),
        # four drafted tokens of one chat, a small vocabulary
        dict(name="verify-chain", op="verify", B=1, n=5, shape="chain", V=32000, q=True),
        # a batch with a draft tree each, a large vocabulary
        dict(name="verify-tree", op="verify", B=16, n=25, shape="tree", V=131072, q=True),
        # a large batch whose drafts were looked up in the prompt (no draft probabilities), an odd vocabulary
        dict(name="verify-lookup", op="verify", B=96, n=6, shape="chain", V=100003, q=False),
        # the accepted path of one chat into the cache, after the last step's tail is cut off
        dict(name="append-path", op="append", B=1, n=8, path=True, layers=10, Hkv=2, D=256, page=64, len=5000,
             dtype="bf16"),
        # a chunk of every prompt of a batch
        dict(name="append-chunk", op="append", B=24, n=500, path=False, layers=10, Hkv=2, D=256, page=64, len=2100,
             dtype="bf16"),
        # one chat branches into four answers, the last four being dropped
        dict(name="fork-small", op="fork", B=1, branches=4, layers=10, Hkv=2, D=256, page=64, len=1500, dtype="bf16"),
        # every chat of a batch branches
        dict(name="fork-batch", op="fork", B=24, branches=4, layers=10, Hkv=2, D=256, page=128, len=3200,
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
    op = rng.choice(["tree", "tree", "tree", "verify", "verify", "append", "fork"])
    while True:
        if op == "tree":
            D = rng.choice([64, 128, 256, 256])
            Hkv = rng.choice([1, 2, 4, 8])
            G = rng.choice([1, 2, 4, 6, 8, 16])
            c = dict(op=op, B=_log(rng, 1, 64), n=_log(rng, 1, 64), shape=rng.choice(["chain", "tree"]), Hq=G * Hkv,
                     Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]), len=_log(rng, 1, 131000),
                     ragged=rng.randrange(6), dtype=rng.choice(["bf16", "bf16", "fp16"]))
            pairs = c["B"] * c["len"] * c["Hq"] * c["n"]
            if c["B"] * c["len"] * Hkv * D > 131000 * 1024 or pairs > 131000 * 16 * 61 or c["Hq"] > 64:
                continue
        elif op == "verify":
            c = dict(op=op, B=_log(rng, 1, 96), n=_log(rng, 2, 32), shape=rng.choice(["chain", "tree"]),
                     V=_log(rng, 1000, 131072), q=rng.random() < 0.7)
            if c["B"] * c["n"] * c["V"] > 96 * 6 * 100003:
                continue
        elif op == "append":
            path = rng.random() < 0.5
            c = dict(op=op, B=_log(rng, 1, 64), n=_log(rng, 1, 64) if path else _log(rng, 1, 500), path=path,
                     layers=rng.choice([1, 4, 10]), Hkv=rng.choice([1, 2, 8]), D=rng.choice([64, 128, 256]),
                     page=rng.choice([16, 32, 64, 128]), len=_log(rng, 1, 4000), dtype=rng.choice(["bf16", "fp16"]))
            if _pool_rows(c) * c["layers"] * c["Hkv"] * c["D"] > 24 * 2700 * 10 * 512:
                continue
        else:
            c = dict(op=op, B=_log(rng, 1, 32), branches=rng.choice([1, 2, 4, 8]), layers=rng.choice([1, 4, 10]),
                     Hkv=rng.choice([1, 2, 8]), D=rng.choice([64, 128, 256]), page=rng.choice([16, 32, 64, 128]),
                     len=_log(rng, 1, 4000), dtype=rng.choice(["bf16", "fp16"]))
            if _pool_rows(c) * c["layers"] * c["Hkv"] * c["D"] > 24 * 4000 * 10 * 512:
                continue
        w = work(c)
        if w["bytes"] <= tops[op][0] and w["flops"] <= tops[op][1]:
            return c


# ---------------------------------------------------- shapes that a case fixes

def _lens(c):
    """Cached tokens per sequence: all of one length, or spread over 1/8 .. 1 of it."""
    if not c.get("ragged"):
        return [c["len"]] * c["B"]
    r = random.Random(c["ragged"])
    return [max(1, int(c["len"] * (1.0 if b == 0 else 0.125 + 0.875 * r.random()))) for b in range(c["B"])]


def _counts(c):
    """Rows or nodes per sequence: up to n, uneven where the case is."""
    if c["op"] == "append":
        return [max(1, c["n"] - (37 * b) % (c["n"] // 2 + 1)) for b in range(c["B"])]
    if c.get("ragged"):
        return [max(1, c["n"] - b % 3) for b in range(c["B"])]
    return [c["n"]] * c["B"]


def _parents(c, n):
    """A draft tree of n nodes: a chain, or levels that narrow as a beam search's do."""
    if c["shape"] == "chain":
        return [i - 1 for i in range(n)]
    return [-1 if i == 0 else 0 if i <= 4 else max(0, (i - 2) // 2 - (i * 7) % 3) for i in range(n)]


def _kept(c, n):
    """Rows an append keeps of n: about half of a path, all of a chunk."""
    return max(1, (n + 1) // 2) if c["path"] else n


def _pages(rows, page):
    return -(-rows // page)


def _pool_rows(c):
    """Rows of the page pool of a case (a quarter of its pages stays free)."""
    if c["op"] == "fork":
        need = c["B"] * (_pages(c["len"], c["page"]) + 2 * c["branches"])
    else:
        need = c["B"] * _pages(c["len"] + c.get("n", 0) * 2, c["page"])
    return (need + need // 4 + 8) * c["page"]


def work(case):
    c = case
    if c["op"] == "tree":
        lens, counts = _lens(c), _counts(c)
        rows = sum(counts)
        seen = 0
        for L, n in zip(lens, counts):
            par, depth = _parents(c, n), []
            for i in range(n):
                depth.append(1 if par[i] < 0 else depth[par[i]] + 1)
            seen += n * L + sum(depth)
        kv = 2 * (sum(lens) + rows) * c["Hkv"] * c["D"] * 2
        return {"bytes": float(kv + 2 * rows * c["Hq"] * c["D"] * 2), "flops": 4.0 * seen * c["Hq"] * c["D"]}
    if c["op"] == "verify":
        # the distributions of the node the walk ends at, and a pair of values for every node passed
        return {"bytes": float(c["B"] * (c["V"] * 4 * (2 if c["q"] else 1) + 24 * c["n"])),
                "flops": float(c["B"] * c["V"] * (3 if c["q"] else 1))}
    row = c["layers"] * c["Hkv"] * c["D"] * 2 * 2
    if c["op"] == "append":
        return {"bytes": float(2 * row * sum(_kept(c, n) for n in _counts(c))), "flops": 0.0}
    tail = sum(L % c["page"] for L in _fork_lens(c))
    return {"bytes": float(2 * row * tail * c["branches"] + c["B"] * c["branches"] * _pages(c["len"], c["page"]) * 12),
            "flops": 0.0}


def _fork_lens(c):
    return [max(1, c["len"] - 29 * b % max(1, c["len"] // 2)) for b in range(c["B"])]


# -------------------------------------------------------------------- inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _offsets(counts):
    return _ints(np.concatenate([[0], np.cumsum(counts)]).tolist())


def _cache(c, g, lens, slots, spare, layers):
    """A page pool and its tables: the first sequences hold `lens` tokens in pages scattered over the pool."""
    page, P = c["page"], _pool_rows(c) // c["page"]
    shape = (layers, P, page, c["Hkv"], c["D"])
    k = torch.empty(shape, dtype=TYPES[c["dtype"]], device=DEV).normal_(generator=g)
    v = torch.empty(shape, dtype=TYPES[c["dtype"]], device=DEV).normal_(generator=g)
    order = torch.randperm(P, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    width = max(_pages(L + spare, page) for L in lens)
    table = torch.full((slots, width), -1, dtype=torch.int32, device=DEV)
    used = [_pages(L, page) for L in lens]
    start = np.concatenate([[0], np.cumsum(used)])
    for b, u in enumerate(used):
        table[b, :u] = order[int(start[b]):int(start[b]) + u]
    refs = torch.zeros(P, dtype=torch.int32, device=DEV)
    refs[order[:int(start[-1])].long()] = 1
    full = torch.zeros(slots, dtype=torch.int32, device=DEV)
    full[:len(lens)] = _ints(lens)
    return dict(k=k, v=v, refs=refs, table=table, lens=full, status=torch.zeros(4, dtype=torch.int32, device=DEV))


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * seed + 17)
    s = {"case": c}

    def normal(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=g)

    if c["op"] == "tree":
        lens, counts = _lens(c), _counts(c)
        N, t = sum(counts), TYPES[c["dtype"]]
        s["cache"] = _cache(c, g, lens, c["B"], 0, 1)
        s["q"] = normal(N, c["Hq"], c["D"], dtype=t)
        s["k_new"] = normal(N, c["Hkv"], c["D"], dtype=t)
        s["v_new"] = normal(N, c["Hkv"], c["D"], dtype=t)
        s["offsets"] = _offsets(counts)
        s["parent"] = _ints([p for n in counts for p in _parents(c, n)])
        s["o"] = torch.zeros_like(s["q"])
    elif c["op"] == "verify":
        B, n, V = c["B"], c["n"], c["V"]
        logits = normal(B * n, V) * 2.5
        draft = logits + normal(B * n, V) * 0.7
        s["p"] = torch.softmax(logits, -1)
        s["q"] = torch.softmax(draft, -1) if c["q"] else None
        par = _parents(c, n)
        s["parent"] = _ints(par * B)
        # every child is drawn from its parent's draft distribution (a looked-up one: mostly the likeliest token)
        src = (torch.arange(B, device=DEV)[:, None] * n + _ints([max(0, p) for p in par]).long()[None]).reshape(-1)
        noise = torch.empty(B * n, V, device=DEV).exponential_(generator=g).log_()
        picked = (draft[src] - noise * (1.0 if c["q"] else 0.2)).argmax(-1)
        s["tokens"] = picked.to(torch.int32)
        s["offsets"] = _offsets([n] * B)
        s["u_accept"] = torch.rand(B * n, generator=g, device=DEV)
        s["u_sample"] = torch.rand(B, generator=g, device=DEV)
        s["path"] = torch.zeros(B, n, dtype=torch.int32, device=DEV)
        s["n_path"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        s["next"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        s["status"] = torch.zeros(4, dtype=torch.int32, device=DEV)
    elif c["op"] == "append":
        counts, t = _counts(c), TYPES[c["dtype"]]
        N = sum(counts)
        lens = [max(1, c["len"] - 13 * b % max(1, c["len"] // 2)) for b in range(c["B"])]
        s["cache"] = _cache(c, g, lens, c["B"], c["n"], c["layers"])
        # what the step before left behind: some of the cached tokens are taken back first
        s["cut"] = _ints([max(0, L - 3) for L in lens])
        s["k_new"] = normal(c["layers"], N, c["Hkv"], c["D"], dtype=t)
        s["v_new"] = normal(c["layers"], N, c["Hkv"], c["D"], dtype=t)
        s["offsets"] = _offsets(counts)
        kept = [_kept(c, n) for n in counts]
        s["n_keep"] = _ints(kept)
        s["path"] = None
        if c["path"]:
            pick = torch.rand(c["B"], c["n"], generator=g, device=DEV)
            pick = torch.where(torch.arange(c["n"], device=DEV)[None] < _ints(counts)[:, None], pick, 2.0)
            order = pick.argsort(-1)
            order = torch.where(torch.arange(c["n"], device=DEV)[None] < s["n_keep"][:, None], order, c["n"])
            s["path"] = order.sort(-1).values.clamp_(max=c["n"] - 1).to(torch.int32).contiguous()
    else:
        lens, m = _fork_lens(c), c["branches"]
        s["cache"] = _cache(c, g, lens, c["B"] * (1 + m), 0, c["layers"])
        s["src"] = torch.arange(c["B"], device=DEV, dtype=torch.int32).repeat_interleave(m).contiguous()
        s["dst"] = c["B"] + torch.arange(c["B"] * m, device=DEV, dtype=torch.int32)
        s["zero"] = torch.zeros(c["B"] * m, dtype=torch.int32, device=DEV)
    if own:
        _handles(s)
    return s


def _handles(s):
    """The cache handle and the workspace that a user's program keeps."""
    import bit_grouped_expert_gb300 as moe
    c = s["case"]
    if "cache" in s:
        k = s["cache"]
        s["handle"] = moe.make_attn_cache(k["k"], k["v"], k["refs"], k["table"], k["lens"], k["status"])
    need = 0
    if c["op"] == "tree":
        need = moe.attn_tree_workspace_bytes(s["handle"], c["B"], s["q"].shape[0], c["n"], c["Hq"])
    elif c["op"] == "append":
        need = moe.attn_cache_append_workspace_bytes(s["handle"], c["B"], s["k_new"].shape[1])
    elif c["op"] == "fork":
        need = moe.attn_cache_fork_workspace_bytes(s["handle"], c["B"] * c["branches"])
    s["ws"] = torch.zeros(max(need, 16), dtype=torch.uint8, device=DEV)


# ----------------------------------------------------------------- the passes

def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    return {"tree": _tree, "verify": _verify, "append": _append, "fork": _fork}[c["op"]](s, c)


def _run_own(s, c):
    import bit_grouped_expert_gb300 as moe
    if c["op"] == "tree":
        moe.attn_tree(s["handle"], 0, s["q"], s["k_new"], s["v_new"], s["offsets"], s["parent"], c["B"], c["n"],
                      s["ws"], s["o"])
        return {"o": s["o"]}
    if c["op"] == "verify":
        moe.moe_draft_verify(s["p"], s["q"], s["tokens"], s["parent"], s["offsets"], s["u_accept"], s["u_sample"],
                             c["B"], s["path"], s["n_path"], s["next"], s["status"])
        return {"path": s["path"], "n_path": s["n_path"], "next": s["next"]}
    if c["op"] == "append":
        moe.attn_cache_trim(s["handle"], None, s["cut"], c["B"])
        moe.attn_cache_append(s["handle"], s["k_new"], s["v_new"], s["offsets"], c["B"], s["ws"], path=s["path"],
                              n_keep=s["n_keep"])
    else:
        moe.attn_cache_trim(s["handle"], s["dst"], s["zero"], c["B"] * c["branches"])
        moe.attn_cache_fork(s["handle"], s["src"], s["dst"], c["B"] * c["branches"], s["ws"])
    return _cache_out(s)


def _cache_out(s):
    return {n: s["cache"][n] for n in ("k", "v", "refs", "table", "lens")}


def _tree(s, c):
    cache, n, Hkv, G, D = s["cache"], c["n"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    B, dt = c["B"], s["q"].dtype
    off = s["offsets"].long()
    i = torch.arange(n, device=DEV)
    real = i[None] < (off[1:] - off[:-1])[:, None]                                   # [B, n]
    rows = (off[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    par = torch.where(real, s["parent"].long()[rows], -2)
    # ancestors and the node itself: (I - P)^-1 = I + P + P^2 + .. of the parent matrix
    P = (par[:, :, None] == i).float()
    eye = torch.eye(n, device=DEV).expand(B, n, n)
    sees = torch.linalg.solve_triangular(eye - P, eye, upper=False, unitriangular=True) > 0.5
    sees = sees & (par > -2)[:, :, None] & real[:, :, None]
    table = cache["table"].long().clamp(min=0)
    L = table.shape[1] * c["page"]
    k = torch.cat([cache["k"][0][table].reshape(B, L, Hkv, D), s["k_new"][rows]], 1).float()
    v = torch.cat([cache["v"][0][table].reshape(B, L, Hkv, D), s["v_new"][rows]], 1).float()
    old = (torch.arange(L, device=DEV)[None] < cache["lens"][:, None])[:, None] & real[:, :, None]
    mask = torch.cat([old & (par > -2)[:, :, None], sees], 2)                        # [B, n, L + n]
    v = torch.where(mask.any(1)[:, :, None, None], v, 0.0)
    q = s["q"][rows].float().reshape(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    a = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(D ** -0.5).reshape(B, Hkv, G, n, L + n)
    a = a.masked_fill_(~mask[:, None, None], float("-inf"))
    a = torch.exp(a - a.amax(-1, keepdim=True).clamp(min=-3e38))
    den = a.sum(-1, keepdim=True)
    o = torch.matmul(a.reshape(B, Hkv, G * n, L + n), v.permute(0, 2, 1, 3)).reshape(B, Hkv, G, n, D)
    o = torch.where(den > 0, o / den, 0.0).permute(0, 3, 1, 2, 4).reshape(B, n, c["Hq"], D)
    return {"o": o[real].to(dt)}


def _verify(s, c):
    B, n, V = c["B"], c["n"], c["V"]
    first = s["offsets"].long()[:-1]
    cur = torch.zeros(B, dtype=torch.int64, device=DEV)
    R, S = s["p"][first].double(), torch.ones(B, dtype=torch.float64, device=DEV)
    path = torch.full((B, n), -1, dtype=torch.int32, device=DEV)
    path[:, 0] = 0
    count = torch.ones(B, dtype=torch.int64, device=DEV)
    for j in range(1, n):  # a child's test rests on the walk before it
        child = s["parent"].long()[first + j] == cur
        x = s["tokens"].long()[first + j][:, None]
        Rx = R.gather(1, x)[:, 0]
        qc = s["q"][first + cur].double() if s["q"] is not None else None
        qx = qc.gather(1, x)[:, 0] if qc is not None else torch.ones_like(S)
        take = child & (s["u_accept"].double()[first + j] * S * qx < Rx)
        drop = child & ~take
        if qc is not None:
            left = (R - S[:, None] * qc).clamp_(min=0.0)
            mass = left.sum(-1)
        else:
            left, mass = R.scatter(1, x, 0.0), S - Rx
        R = torch.where(take[:, None], s["p"][first + j].double(), torch.where(drop[:, None], left, R))
        S = torch.where(take, 1.0, torch.where(drop, mass, S))
        cur = torch.where(take, j, cur)
        slot = torch.where(take, count, n)
        path = torch.cat([path, path[:, :1]], 1).scatter_(1, slot[:, None], j)[:, :n]
        count = count + take
    sums = R.cumsum(-1)
    empty = ~(sums[:, -1] > 0)
    sums = torch.where(empty[:, None], s["p"][first + cur].double().cumsum(-1), sums)
    last = sums[:, -1:]
    want = s["u_sample"].double()[:, None] * last
    nxt = torch.minimum((sums <= want).sum(-1), (sums < last).sum(-1))
    return {"path": path, "n_path": count.to(torch.int32), "next": nxt.to(torch.int32)}


def _trim(cache, slots, new, page):
    table = cache["table"][slots]
    j = torch.arange(table.shape[1], device=DEV)[None]
    gone = (j >= ((new + page - 1) // page)[:, None]) & (table >= 0)
    cache["refs"].index_add_(0, table.clamp(min=0).reshape(-1), -gone.reshape(-1).to(torch.int32))
    cache["table"][slots] = torch.where(gone, -1, table)
    cache["lens"][slots] = new


def _free_pages(cache):
    return torch.sort((cache["refs"] != 0).to(torch.uint8), stable=True).indices.to(torch.int32)


def _append(s, c):
    cache, page, B = s["cache"], c["page"], c["B"]
    slots = torch.arange(B, device=DEV)
    _trim(cache, slots, s["cut"], page)
    old, keep = cache["lens"], s["n_keep"]
    have, want = (old + page - 1) // page, (old + keep + page - 1) // page
    need = want - have
    first = need.cumsum(0) - need
    free = _free_pages(cache)
    j = torch.arange(cache["table"].shape[1], device=DEV)[None]
    new = (j >= have[:, None]) & (j < want[:, None])
    pages = free[(first[:, None] + j - have[:, None]).clamp(min=0, max=free.numel() - 1).long()]
    cache["table"].copy_(torch.where(new, pages, cache["table"]))
    cache["refs"].index_add_(0, torch.where(new, pages, 0).reshape(-1), new.reshape(-1).to(torch.int32))
    i = torch.arange(c["n"], device=DEV)[None]
    i = torch.minimum(i, (keep - 1)[:, None])                  # rows past the kept ones repeat the last of them
    row = s["path"].gather(1, i.long()) if s["path"] is not None else i
    src = (s["offsets"][:-1, None] + row).reshape(-1)
    pos = old[:, None] + i
    dst = (cache["table"].gather(1, (pos // page).long()) * page + pos % page).reshape(-1).long()
    for pool, rows in ((cache["k"], s["k_new"]), (cache["v"], s["v_new"])):
        pool.view(c["layers"], -1, c["Hkv"], c["D"])[:, dst] = rows[:, src]
    cache["lens"].add_(keep)
    return _cache_out(s)


def _fork(s, c):
    cache, page = s["cache"], c["page"]
    src, dst = s["src"].long(), s["dst"].long()
    _trim(cache, dst, s["zero"], page)
    L = cache["lens"][src]
    full, rest = L // page, L % page
    part = (rest > 0).to(torch.int32)
    free = _free_pages(cache)
    fresh = free[(part.cumsum(0) - part).long()]
    table = cache["table"][src]
    j = torch.arange(table.shape[1], device=DEV)[None]
    shared = j < full[:, None]
    cache["refs"].index_add_(0, table.clamp(min=0).reshape(-1), shared.reshape(-1).to(torch.int32))
    cache["refs"].index_add_(0, fresh, part)
    cache["table"][dst] = torch.where(shared, table, torch.where((j == full[:, None]) & (part > 0)[:, None],
                                                                 fresh[:, None], -1))
    cache["lens"][dst] = L
    old = table.gather(1, full[:, None].clamp(max=table.shape[1] - 1).long())[:, 0].clamp(min=0)
    r = torch.arange(page, device=DEV)
    r = torch.minimum(r[None], (rest - 1).clamp(min=0)[:, None])   # rows past the last repeat it
    to = torch.where(part > 0, fresh, old)                          # nothing to copy: onto itself
    at, put = (old[:, None] * page + r).reshape(-1).long(), (to[:, None] * page + r).reshape(-1).long()
    for pool in (cache["k"], cache["v"]):
        flat = pool.view(c["layers"], -1, c["Hkv"], c["D"])
        flat[:, put] = flat[:, at]
    return _cache_out(s)


# ------------------------------------------------------- values in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"tree": _exact_tree, "verify": _exact_verify, "append": _exact_pages, "fork": _exact_pages}[case["op"]](s, case)


def _exact_tree(s, c):
    if work(c)["flops"] > 3e11:
        return None
    off, par = s["offsets"].tolist(), s["parent"].tolist()
    lens, page, G = s["cache"]["lens"].tolist(), c["page"], c["Hq"] // c["Hkv"]
    out = []
    for b in range(c["B"]):
        lo, hi, L = off[b], off[b + 1], lens[b]
        pages = s["cache"]["table"][b].long()[:_pages(L, page)]
        for_all = {}
        for name in ("k", "v"):
            old = s["cache"][name][0].index_select(0, pages).reshape(-1, c["Hkv"], c["D"])[:L]
            for_all[name] = torch.cat([old, s[name + "_new"][lo:hi]]).double()
        line = np.zeros((hi - lo, hi - lo), bool)
        for i in range(hi - lo):
            a = i
            while a >= 0:
                line[i, a] = True
                a = par[lo + a]
        see = torch.cat([torch.ones(hi - lo, L, dtype=torch.bool, device=DEV), torch.from_numpy(line).to(DEV)], 1)
        o = torch.empty(hi - lo, c["Hq"], c["D"], dtype=torch.float64, device=DEV)
        for h in range(c["Hq"]):
            a = (s["q"][lo:hi, h].double() @ for_all["k"][:, h // G].T) / np.sqrt(c["D"])
            a[~see] = -np.inf
            o[:, h] = torch.softmax(a, -1) @ for_all["v"][:, h // G]
        out.append(o)
    return {"o": torch.cat(out)}


def _exact_verify(s, c):
    B, n = c["B"], c["n"]
    path, count, nxt = np.full((B, n), -1, np.int64), [], []
    par, tok = s["parent"].cpu().numpy().reshape(B, n), s["tokens"].cpu().numpy().reshape(B, n)
    ua, us = s["u_accept"].double().cpu().numpy().reshape(B, n), s["u_sample"].double().cpu().numpy()

    def row(name, b, i):
        return s[name][b * n + i].double().cpu().numpy()

    for b in range(B):
        at, steps, mass, rest = 0, [0], 1.0, row("p", b, 0)
        draft = row("q", b, 0) if c["q"] else None
        for j in range(1, n):
            if par[b, j] != at:
                continue
            x = tok[b, j]
            if ua[b, j] * mass * (draft[x] if c["q"] else 1.0) < rest[x]:
                at, mass, rest = j, 1.0, row("p", b, j)
                draft = row("q", b, j) if c["q"] else None
                steps.append(j)
            elif c["q"]:
                rest = np.maximum(rest - mass * draft, 0.0)
                mass = rest.sum()
            else:
                mass -= rest[x]
                rest[x] = 0.0
        if not rest.sum() > 0:
            rest = row("p", b, at)
        sums = np.cumsum(rest)
        nxt.append(min(int(np.searchsorted(sums, us[b] * sums[-1], side="right")), int(np.flatnonzero(rest)[-1])))
        path[b, :len(steps)] = steps
        count.append(len(steps))
    return {"path": torch.from_numpy(path), "n_path": torch.tensor(count), "next": torch.tensor(nxt)}


def _exact_pages(s, c):
    cache, page = s["cache"], c["page"]
    refs, table, lens = (cache[n].cpu().numpy().copy() for n in ("refs", "table", "lens"))
    cut = zip(range(c["B"]), s["cut"].tolist()) if c["op"] == "append" else ((d, 0) for d in s["dst"].tolist())
    for slot, new in cut:
        for j in range(_pages(new, page), table.shape[1]):
            if table[slot, j] >= 0:
                refs[table[slot, j]] -= 1
                table[slot, j] = -1
        lens[slot] = new
    free = iter(np.flatnonzero(refs == 0).tolist())
    if c["op"] == "append":
        off, keep = s["offsets"].tolist(), s["n_keep"].tolist()
        path = s["path"].tolist() if s["path"] is not None else None
        src, dst = [], []
        for b in range(c["B"]):
            for i in range(keep[b]):
                if lens[b] % page == 0:
                    table[b, lens[b] // page] = page_id = next(free)
                    refs[page_id] = 1
                src.append(off[b] + (path[b][i] if path else i))
                dst.append(int(table[b, lens[b] // page]) * page + int(lens[b]) % page)
                lens[b] += 1
        pairs = [(cache[n], s[n + "_new"]) for n in ("k", "v")]
    else:
        src, dst = [], []
        for a, d in zip(s["src"].tolist(), s["dst"].tolist()):
            whole, rest = divmod(int(lens[a]), page)
            table[d, :whole] = table[a, :whole]
            refs[table[a, :whole]] += 1
            if rest:
                table[d, whole] = page_id = next(free)
                refs[page_id] = 1
                src += [int(table[a, whole]) * page + r for r in range(rest)]
                dst += [page_id * page + r for r in range(rest)]
            lens[d] = lens[a]
        pairs = [(cache[n], cache[n].clone().view(c["layers"], -1, c["Hkv"], c["D"])) for n in ("k", "v")]
    src, dst = torch.tensor(src, device=DEV), torch.tensor(dst, device=DEV)
    for pool, rows in pairs:
        if src.numel():
            pool.view(c["layers"], -1, c["Hkv"], c["D"])[:, dst] = rows[:, src]
    return {"k": cache["k"].double(), "v": cache["v"].double(), "refs": torch.from_numpy(refs),
            "table": torch.from_numpy(table), "lens": torch.from_numpy(lens)}
