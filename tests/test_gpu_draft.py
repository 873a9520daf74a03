"""GPU parity of draft verification (moe_draft_verify) against the fp64 oracle:
paths and tokens exactly, and a run of the operators together as a speculative
decoding step uses them."""
from __future__ import annotations

import numpy as np
import pytest

from oracle.tree import Pages, tree_attention, verify_drafts

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import bit_grouped_expert_gb300 as moe  # noqa: E402

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_grouped_expert_gb300 import build
    build.build()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def verify(p, q, tokens, parent, off, ua, us, stride, stream=None, status=None):
    B = len(off) - 1
    path = torch.full((B, stride), 99, dtype=torch.int32, device=DEV)
    n, nxt = i32([99] * B), i32([99] * B)
    status = torch.zeros(4, dtype=torch.int32, device=DEV) if status is None else status
    f = lambda a: torch.as_tensor(np.asarray(a, np.float32), device=DEV)  # noqa: E731
    moe.moe_draft_verify(f(p), None if q is None else f(q), i32(list(tokens)), i32(list(parent)), i32(list(off)), f(ua), f(us),
                         B, path, n, nxt, status, stream=stream)
    torch.cuda.synchronize()
    return path.cpu().numpy(), n.tolist(), nxt.tolist(), int(status[0])


def probs(r, n, V, heat=2.5):
    x = np.exp(r.normal(0, heat, (n, V)))
    return (x / x.sum(-1, keepdims=True)).astype(np.float32)


def trees(r, B, most):
    out = []
    for _ in range(B):
        n = int(r.integers(1, most + 1))
        out.append([-1] + [int(r.integers(max(0, i - 4), i)) if r.random() > 0.1 else -2 for i in range(1, n)])
    return [[p if p < 0 or t[p] != -2 else -2 for p in t] for t in out]


def same(got, p, q, tokens, parents, off, ua, us):
    path, n, nxt, status = got
    assert status == 0
    for b, par in enumerate(parents):
        s = slice(off[b], off[b + 1])
        want, token = verify_drafts(p[s], None if q is None else q[s], tokens[s], par, ua[s], us[b])
        assert n[b] == len(want) and path[b, :n[b]].tolist() == want and (path[b, n[b]:] == -1).all()
        assert nxt[b] == token, (b, nxt[b], token)


@pytest.mark.parametrize("V", [1, 2, 5, 31, 32, 33, 255, 1000, 1023, 4097, 32000, 100003])
@pytest.mark.parametrize("drafted", [True, False])
def test_vocabularies(V, drafted):
    r = np.random.default_rng(V)
    parents = trees(r, 6, 9)
    off = np.concatenate([[0], np.cumsum([len(t) for t in parents])])
    N = int(off[-1])
    p = probs(r, N, V)
    q = np.abs(p + 0.5 * probs(r, N, V)) if drafted else None
    if drafted:
        q = (q / q.sum(-1, keepdims=True)).astype(np.float32)
    tokens = np.array([int(r.choice(V, p=p[i].astype(np.float64) / p[i].astype(np.float64).sum())) for i in range(N)])
    ua, us = r.random(N, dtype=np.float32), r.random(6, dtype=np.float32)
    same(verify(p, q, tokens, [x for t in parents for x in t], off, ua, us, 9), p, q, tokens, parents, off, ua, us)


@pytest.mark.parametrize("B,most,seed", [(1, 64, 0), (200, 12, 1), (40, 33, 2)])
@pytest.mark.parametrize("drafted", [True, False])
def test_many_trees(B, most, seed, drafted):
    r = np.random.default_rng(seed)
    V = 700
    parents = trees(r, B, most)
    off = np.concatenate([[0], np.cumsum([len(t) for t in parents])])
    N = int(off[-1])
    p = probs(r, N, V, 1.0)
    q = probs(r, N, V, 1.0) if drafted else None
    tokens = r.integers(0, 40, N)
    ua, us = (r.random(N, dtype=np.float32) * 0.3).astype(np.float32), r.random(B, dtype=np.float32)
    same(verify(p, q, tokens, [x for t in parents for x in t], off, ua, us, most), p, q, tokens, parents, off, ua, us)


@pytest.mark.parametrize("B", [1, 20, 25, 34, 43, 60, 100, 152, 153, 400])
def test_clusters_of_all_sizes(B):
    # from 16 CTAs a tree down to one
    r = np.random.default_rng(B)
    V, n = 17000, 3
    p, q = probs(r, n * B, V, 1.0), probs(r, n * B, V, 1.0)
    tokens, parents = r.integers(0, V, n * B), [[-1, 0, 0]] * B
    off = [n * b for b in range(B + 1)]
    ua, us = (r.random(n * B, dtype=np.float32) + np.float32(0.5)) % np.float32(1), r.random(B, dtype=np.float32)
    for d in (q, None):
        same(verify(p, d, tokens, [-1, 0, 0] * B, off, ua, us, n), p, d, tokens, parents, off, ua, us)


def test_long_chains_that_are_taken_whole():
    r = np.random.default_rng(5)
    n, V = 1024, 50
    p = probs(r, n, V)
    tokens = p.argmax(-1)
    tokens = np.concatenate([[0], tokens[:-1]])
    ua = np.zeros(n, np.float32)
    parents = [list(range(-1, n - 1))]
    same(verify(p, p, tokens, parents[0], [0, n], ua, [0.5], n), p, p, tokens, parents, [0, n], ua, np.array([0.5], np.float32))


def test_many_refused_siblings():
    # a root with 63 children of one token each: all refused, the residual shrinks step by step
    r = np.random.default_rng(6)
    n, V = 64, 3000
    p, q = probs(r, n, V, 1.0), probs(r, n, V, 0.2)
    tokens, parents = r.integers(0, V, n), [[-1] + [0] * (n - 1)]
    ua = np.full(n, 0.999, np.float32)
    for d in (q, None):
        same(verify(p, d, tokens, parents[0], [0, n], ua, [0.7], n), p, d, tokens, parents, [0, n], ua, np.array([0.7], np.float32))


def test_draws_at_the_ends():
    p = np.array([[0.0, 0.25, 0.0, 0.75, 0.0]], np.float32)
    big = np.nextafter(np.float32(1), np.float32(0))
    for u, want in ((0.0, 1), (0.25, 3), (0.2499999, 1), (big, 3)):
        got = verify(p, None, [0], [-1], [0, 1], [0.0], [u], 1)
        assert got[2] == [want] and got[3] == 0


def test_the_last_token_may_be_refused_twice():
    # both children carry token 2; once refused its residual is zero, so the second cannot be taken
    p = np.array([[0.2, 0.3, 0.5]] * 3, np.float32)
    got = verify(p, None, [0, 2, 2], [-1, 0, 0], [0, 3], [0, 0.9, 0.0], [0.99], 3)
    assert got[1] == [1] and got[2] == [1]


def test_no_residual_falls_back_to_the_target():
    # p = q and the child's token has no probability: refused, and max(p - q, 0) is zero everywhere
    p = np.array([[0.5, 0.5, 0.0]] * 2, np.float32)
    got = verify(p, p, [0, 2], [-1, 0], [0, 2], [0, 0.0], [0.6], 2)
    assert got[1] == [1] and got[2] == [1] and got[3] == 0


@pytest.mark.parametrize("row", [np.zeros(7), np.full(7, np.nan), np.array([0, 0, np.inf, 0, 0, 0, 0.5])])
def test_no_mass_to_draw_from(row):
    p = np.stack([probs(np.random.default_rng(0), 1, 7)[0], row]).astype(np.float32)
    path, n, nxt, status = verify(p, None, [0, 0], [-1, -1], [0, 1, 2], [0, 0], [0.5, 0.5], 2)
    assert status == moe.MOE_ERR_NONFINITE and n == [1, 0] and nxt[1] == -1 and nxt[0] >= 0 and (path[1] == -1).all()


@pytest.mark.parametrize("change", [dict(tokens=[0, 5]), dict(tokens=[0, -1]), dict(parent=[-1, 1]), dict(parent=[0, 0]),
                                    dict(parent=[-1, -3]), dict(off=[0, 3]), dict(off=[-1, 2]), dict(off=[2, 0]),
                                    dict(stride=1)])
def test_device_checks(change):
    a = {**dict(tokens=[0, 1], parent=[-1, 0], off=[0, 2], stride=2), **change}
    p = probs(np.random.default_rng(0), 2, 5)
    path, n, nxt, status = verify(p, None, a["tokens"], a["parent"], a["off"], [0, 0], [0.5], a["stride"])
    assert status == moe.MOE_ERR_DEVICE_BOUNDS and n == [0] and nxt == [-1] and (path == -1).all()


def test_empty_trees():
    p = probs(np.random.default_rng(0), 2, 5)
    path, n, nxt, status = verify(p, None, [0, 1], [-1, 0], [0, 0, 2, 2], [0, 0], [0.1, 0.2, 0.3], 2)
    assert status == 0 and n[0] == n[2] == 0 and nxt[0] == nxt[2] == -1 and n[1] >= 1


def test_replays_from_a_graph_on_another_stream():
    r = np.random.default_rng(9)
    n, V = 5, 9000
    p, q = (torch.from_numpy(probs(r, n, V)).to(DEV) for _ in range(2))
    tok, par, off = i32(r.integers(0, V, n).tolist()), i32([-1, 0, 1, 2, 3]), i32([0, n])
    ua, us = torch.zeros(n, device=DEV), torch.zeros(1, device=DEV)
    path, cnt, nxt, st = i32([[0] * n]), i32([0]), i32([0]), i32([0, 0, 0, 0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            moe.moe_draft_verify(p, q, tok, par, off, ua, us, 1, path, cnt, nxt, st)
    for i in range(4):
        ua.copy_(torch.from_numpy(r.random(n, dtype=np.float32)))
        us.fill_(0.2 * i + 0.1)
        g.replay()
        torch.cuda.synchronize()
        want, token = verify_drafts(p.cpu().numpy(), q.cpu().numpy(), tok.tolist(), par.tolist(), ua.tolist(),
                                    float(us))
        assert path[0, :int(cnt)].tolist() == want and int(nxt) == token


def test_a_speculative_decoding_run():
    """Prompts, a fork, then steps of tree attention, verification and append on
    two layers, against the oracles after every step."""
    r = np.random.default_rng(11)
    layers, Hq, Hkv, D, page, V, n = 2, 16, 2, 128, 16, 500, 6
    k = torch.zeros(layers, 64, page, Hkv, D, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    refs, lens = i32([0] * 64), i32([0] * 4)
    table, status = torch.full((4, 16), -1, dtype=torch.int32, device=DEV), i32([0] * 4)
    cache = moe.make_attn_cache(k, v, refs, table, lens, status)
    model = Pages(k.float().cpu().numpy(), v.float().cpu().numpy(),
                  *[t.cpu().numpy().copy() for t in (refs, table, lens)])

    def rows(m):
        return [torch.from_numpy(r.normal(size=(layers, m, Hkv, D)).astype(np.float32)).to(DEV).bfloat16() for _ in range(2)]

    pk, pv = rows(30)
    ws = torch.empty(max(moe.attn_cache_append_workspace_bytes(cache, 4, 64), moe.attn_cache_fork_workspace_bytes(cache, 2),
                         moe.attn_tree_workspace_bytes(cache, 4, 4 * n, n, Hq)), dtype=torch.uint8, device=DEV)
    moe.attn_cache_append(cache, pk, pv, i32([0, 21, 30]), 2, ws)
    moe.attn_cache_fork(cache, i32([0, 1]), i32([2, 3]), 2, ws)
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    model.append([(0, f(pk[:, :21]), f(pv[:, :21])), (1, f(pk[:, 21:]), f(pv[:, 21:]))])
    model.fork([(0, 2), (1, 3)])
    parent = [-1, 0, 0, 1, 1, 2]
    off = [b * n for b in range(5)]
    path, cnt, nxt = torch.zeros(4, n, dtype=torch.int32, device=DEV), i32([0] * 4), i32([0] * 4)
    taken = 0
    for _ in range(8):
        kn, vn = rows(4 * n)
        for layer in range(layers):
            q = torch.from_numpy(r.normal(size=(4 * n, Hq, D)).astype(np.float32)).to(DEV).bfloat16()
            o = torch.empty_like(q)
            moe.attn_tree(cache, layer, q, kn[layer], vn[layer], i32(off), i32(parent * 4), 4, n, ws, o)
            for b in range(4):
                ko, vo = model.rows(b, layer)
                s = slice(b * n, b * n + n)
                ref = tree_attention(f(q[s]), ko, vo, f(kn[layer, s]), f(vn[layer, s]), parent)[0]
                assert np.linalg.norm(f(o[s]) - ref) <= 2 * 2.0 ** -8 * np.linalg.norm(ref)
        p, d = probs(r, 4 * n, V, 1.0), probs(r, 4 * n, V, 1.0)
        tokens = np.array([int(r.choice(V, p=d[b * n + max(0, parent[i])] / d[b * n + max(0, parent[i])].astype(np.float64).sum()))
                           for b in range(4) for i in range(n)])
        ua, us = r.random(4 * n, dtype=np.float32), r.random(4, dtype=np.float32)
        t = lambda a: torch.from_numpy(np.asarray(a)).to(DEV)  # noqa: E731
        moe.moe_draft_verify(t(p), t(d), t(tokens.astype(np.int32)), i32(parent * 4), i32(off), t(ua), t(us), 4, path, cnt, nxt,
                             status)
        moe.attn_cache_append(cache, kn, vn, i32(off), 4, ws, path=path, n_keep=cnt)
        jobs = []
        for b in range(4):
            s = slice(b * n, b * n + n)
            want, token = verify_drafts(p[s], d[s], tokens[s], parent, ua[s], us[b])
            assert path[b, :int(cnt[b])].tolist() == want and int(nxt[b]) == token
            pick = [b * n + i for i in want]
            taken += len(want) - 1
            jobs.append((b, f(kn)[:, pick], f(vn)[:, pick]))
        model.append(jobs)
        for a, m in ((refs, model.refs), (table, model.table), (lens, model.lens)):
            np.testing.assert_array_equal(a.cpu().numpy(), m)
        np.testing.assert_array_equal(f(k), model.k)
        np.testing.assert_array_equal(f(v), model.v)
    assert taken > 0 and int(status[0]) == 0


def refusals(B, V, kids):
    """B trees of a root with `kids` children that are all refused (u = 0.999 and p below q at their tokens),
    p and q everywhere positive and finite."""
    r = np.random.default_rng(31)
    n = kids + 1
    p, q = probs(r, B * n, V, 1.0), probs(r, B * n, V, 1.0)
    tokens = np.zeros(B * n, np.int64)
    for b in range(B):
        tokens[b * n + 1:(b + 1) * n] = np.argsort(p[b * n] / q[b * n])[:kids]
    return p, q, tokens, [-1] + [0] * kids, [n * b for b in range(B + 1)], np.full(B * n, 0.999, np.float32)


# the residual kept in shared memory (one CTA, and a cluster), and rebuilt in every pass (one CTA a tree, a long row)
RESIDUALS = [(3, 500), (3, 20000), (160, 12000)]


@pytest.mark.parametrize("B,V", RESIDUALS)
@pytest.mark.parametrize("kids", [1, 2, 4])
@pytest.mark.parametrize("where,value", [("p", float("nan")), ("p", float("inf")), ("q", float("nan"))])
def test_no_draw_from_a_residual_that_is_not_a_number(B, V, kids, where, value):
    p, q, tokens, tree, off, ua = refusals(B, V, kids)
    us = np.full(B, 0.5, np.float32)
    same(verify(p, q, tokens, tree * B, off, ua, us, kids + 1), p, q, tokens, [tree] * B, off, ua, us)
    at = [t for t in range(V) if t not in tokens[off[1] + 1:off[2]]][3]
    (p if where == "p" else q)[off[1], at] = value  # the second tree's root, at no child's token
    path, n, nxt, status = verify(p, q, tokens, tree * B, off, ua, us, kids + 1)
    assert status == moe.MOE_ERR_NONFINITE and n[1] == 0 and nxt[1] == -1 and (path[1] == -1).all()
    for b in [x for x in range(B) if x != 1][:20]:
        s = slice(off[b], off[b + 1])
        assert nxt[b] == verify_drafts(p[s], q[s], tokens[s], tree, ua[s], us[b])[1] and n[b] == 1


@pytest.mark.parametrize("B,V", RESIDUALS)
def test_a_draft_of_nothing_but_nan_is_not_read_as_no_residual(B, V):
    p, q, tokens, tree, off, ua = refusals(B, V, 2)
    q[0] = np.nan
    path, n, nxt, status = verify(p, q, tokens, tree * B, off, ua, np.full(B, 0.5, np.float32), 3)
    assert status == moe.MOE_ERR_NONFINITE and n[0] == 0 and nxt[0] == -1 and n[1] == 1


@pytest.mark.parametrize("B,V", RESIDUALS)
@pytest.mark.parametrize("kids", [1, 2, 4])
def test_an_infinite_draft_probability_leaves_its_token_nothing(B, V, kids):
    # max(R - S inf, 0) = 0, in every round
    p, q, tokens, tree, off, ua = refusals(B, V, kids)
    us = np.full(B, 0.5, np.float32)
    q[0, :V // 2:2] = np.inf
    same(verify(p, q, tokens, tree * B, off, ua, us, kids + 1), p, q, tokens, [tree] * B, off, ua, us)


@pytest.mark.parametrize("B,V", RESIDUALS)
def test_a_child_of_probability_nan_is_reported_without_draft_probabilities_too(B, V):
    p, _, tokens, tree, off, ua = refusals(B, V, 3)
    p[0, tokens[2]] = np.nan
    path, n, nxt, status = verify(p, None, tokens, tree * B, off, ua, np.full(B, 0.5, np.float32), 4)
    assert status == moe.MOE_ERR_NONFINITE and n[0] == 0 and nxt[0] == -1 and (path[0] == -1).all()
    s = slice(off[1], off[2])
    want, token = verify_drafts(p[s], None, tokens[s], tree, ua[s], 0.5)
    assert path[1, :n[1]].tolist() == want and nxt[1] == token


def test_host_threads_with_vocabularies_of_their_own():
    """Each thread's calls want another amount of shared memory for the residual: none may be refused because of another's."""
    import ctypes
    import threading
    r = np.random.default_rng(34)
    jobs, failed = [], []
    for V in (900, 130000, 9000, 70000):
        n = 3
        p, q = (torch.from_numpy(probs(r, n, V, 1.0)).to(DEV) for _ in range(2))
        ins = p, q, i32([0, 1, 2]), i32([-1, 0, 0]), i32([0, n]), torch.full((n,), 0.999, device=DEV), \
            torch.full((1,), 0.3, device=DEV)
        outs = torch.zeros(1, n, dtype=torch.int32, device=DEV), i32([0]), i32([0]), i32([0, 0, 0, 0])
        want = verify_drafts(p.cpu().numpy(), q.cpu().numpy(), [0, 1, 2], [-1, 0, 0], ins[5].tolist(), float(ins[6]))
        jobs.append((V, ins, outs, torch.cuda.Stream(), want))
    torch.cuda.synchronize()
    call = moe.lib().moe_draft_verify

    def loop(V, ins, outs, stream, want):
        a = [ctypes.c_void_p(t.data_ptr()) for t in ins]
        o = [ctypes.c_void_p(t.data_ptr()) for t in outs]
        args = (*a, 1, 3, V, o[0], 3, *o[1:], ctypes.c_void_p(stream.cuda_stream))
        codes = [call(*args) for _ in range(20000)]
        failed.extend((V, c) for c in codes if c != moe.MOE_OK)

    threads = [threading.Thread(target=loop, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, f"{len(failed)} of 80000 calls refused, the first {failed[0]}"
    for V, ins, outs, stream, want in jobs:
        path, cnt, nxt, st = (t.flatten().tolist() for t in outs)
        assert st[0] == 0 and path[:cnt[0]] == want[0] and nxt[0] == want[1]


@pytest.mark.parametrize("B,run", [(300, 128), (19, 1024)])
def test_a_threshold_between_two_halves_never_picks_a_run_without_mass(B, run):
    """Runs 0 .. 6 hold values of many sizes, runs 7 and 8 nothing, runs 9 .. 15 the values of the first in
    another order: with u = 1/2 the threshold is the sum of the first half, and sums of another order differ from it in
    their last bits.  (A run is a warp's part of the row with one CTA a tree, a CTA's with sixteen.)"""
    r = np.random.default_rng(33)
    V = 16 * run
    p = np.zeros((B, V), np.float32)
    for b in range(B):
        half = (r.random(7 * run) * 2.0 ** -r.uniform(10, 40, 7 * run)).astype(np.float32)
        p[b, :7 * run], p[b, 9 * run:] = half, r.permutation(half)
    path, n, nxt, status = verify(p, None, [0] * B, [-1] * B, range(B + 1), np.zeros(B), np.full(B, 0.5), 1)
    assert status == 0 and n == [1] * B
    for b, t in enumerate(nxt):
        assert t >= 0 and p[b, t] > 0
        sums, half = np.cumsum(p[b].astype(np.float64)), p[b, :7 * run].astype(np.float64).sum()
        assert sums[t] > half * (1 - 2.0 ** -40) and sums[t] - p[b, t] < half * (1 + 2.0 ** -40)


@pytest.mark.parametrize("V", [1 << 20, (1 << 20) - 1])
@pytest.mark.parametrize("drafted", [True, False])
def test_the_largest_vocabularies(V, drafted):
    r = np.random.default_rng(36)
    p, q = probs(r, 4, V, 1.0), probs(r, 4, V, 1.0)
    tokens, tree = [0, V - 1, 7, V // 2], [-1, 0, 0, 0]
    ua, us = np.full(4, 0.9, np.float32), np.array([0.6], np.float32)
    for u in (0.0, 0.6, float(np.nextafter(np.float32(1), np.float32(0)))):
        us[0] = u
        same(verify(p, q if drafted else None, tokens, tree, [0, 4], ua, us, 4), p, q if drafted else None,
             np.array(tokens), [tree], [0, 4], ua, us)


def test_the_most_trees():
    r = np.random.default_rng(37)
    B, V = 65535, 3
    p, q = probs(r, B, V, 1.0), probs(r, B, V, 1.0)
    us = r.random(B, dtype=np.float32)
    path, n, nxt, status = verify(p, q, np.zeros(B, int), [-1] * B, range(B + 1), np.zeros(B), us, 1)
    sums = np.cumsum(p.astype(np.float64), 1)
    assert status == 0 and (path == 0).all() and n == [1] * B
    np.testing.assert_array_equal(nxt, (sums <= us[:, None].astype(np.float64) * sums[:, -1:]).sum(1))


def test_captures_with_copies_and_events_around_the_calls():
    """A copy and a fill as graph nodes directly in front of every entry point, and a call on a forked branch of the
    capture: what a dependent launch waits for is then no kernel, or several nodes."""
    r = np.random.default_rng(35)
    Hq, Hkv, D, V, n = 8, 2, 64, 3000, 4
    k, v = (torch.from_numpy(r.normal(size=(1, 16, 16, Hkv, D)).astype(np.float32)).to(DEV).bfloat16() for _ in range(2))
    refs, table, lens, st = i32([1, 1] + [0] * 14), i32([[0, 1, -1, -1], [-1] * 4, [-1] * 4]), i32([20, 0, 0]), i32([0] * 4)
    cache = moe.make_attn_cache(k, v, refs, table, lens, st)
    first = [t.clone() for t in (k, v, refs, table, lens)]
    kn, vn, q = (torch.from_numpy(r.normal(size=s).astype(np.float32)).to(DEV).bfloat16()
                 for s in ((1, n, Hkv, D), (1, n, Hkv, D), (n, Hq, D)))
    parent, off = [-1, 0, 0, 1], i32([0, n])
    p, d = probs(r, n, V), probs(r, n, V)
    tok, ua, us = [0, 5, 9, 2], r.random(n, dtype=np.float32), np.array([0.4], np.float32)
    pg, dg, uag, usg = (torch.from_numpy(x).to(DEV) for x in (p, d, ua, us))
    hq, hp, par, tokg = q.clone(), pg.clone(), i32(parent), i32(tok)
    path, cnt, nxt = i32([[0] * n]), i32([0]), i32([0])
    o, o2 = torch.empty_like(q), torch.empty_like(q)
    ws = [torch.empty(max(moe.attn_tree_workspace_bytes(cache, 1, n, n, Hq), moe.attn_cache_append_workspace_bytes(cache, 1, n),
                          moe.attn_cache_fork_workspace_bytes(cache, 1)), dtype=torch.uint8, device=DEV) for _ in range(2)]
    src, dst, zero, one = i32([0]), i32([2]), i32([0]), i32([2])
    s, side = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        q.copy_(hq)
        o.zero_()
        moe.attn_tree(cache, 0, q, kn[0], vn[0], off, par, 1, n, ws[0], o)
        o2.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            moe.attn_tree(cache, 0, q, kn[0], vn[0], off, par, 1, n, ws[1], o2)
        pg.copy_(hp)
        path.zero_()
        moe.moe_draft_verify(pg, dg, tokg, par, off, uag, usg, 1, path, cnt, nxt, st)
        torch.cuda.current_stream().wait_stream(side)
        moe.attn_cache_append(cache, kn, vn, off, 1, ws[0], path=path, n_keep=cnt)
        src.copy_(zero)
        moe.attn_cache_fork(cache, src, dst, 1, ws[0])
        dst.copy_(one)
        moe.attn_cache_trim(cache, dst, zero, 1)

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    for _ in range(3):
        for t, old in zip((k, v, refs, table, lens), first):
            t.copy_(old)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        model = Pages(*[x.float().cpu().numpy() for x in first[:2]], *[x.cpu().numpy().copy() for x in first[2:]])
        ref = tree_attention(f(q), *model.rows(0), f(kn[0]), f(vn[0]), parent)[0]
        assert np.linalg.norm(f(o) - ref) <= 2 * 2.0 ** -8 * np.linalg.norm(ref) and torch.equal(o, o2)
        want, token = verify_drafts(p, d, tok, parent, ua, us[0])
        assert path[0, :int(cnt)].tolist() == want and int(nxt) == token
        model.append([(0, f(kn)[:, want], f(vn)[:, want])])
        model.fork([(0, 2)])
        model.trim(2, 0)
        for a, m in ((refs, model.refs), (table, model.table), (lens, model.lens)):
            np.testing.assert_array_equal(a.cpu().numpy(), m)
        np.testing.assert_array_equal(f(k), model.k)
        assert st.tolist() == [0] * 4
