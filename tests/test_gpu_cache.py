"""GPU parity of the paged cache's calls (append, fork, trim) against the
oracle: tables, holder counts, lengths and every row, exactly."""
from __future__ import annotations

import numpy as np
import pytest

from oracle.tree import Pages

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


class Twin:
    """A cache on the GPU and the oracle's copy of it; check() holds one against the other."""

    def __init__(self, pages=40, page=16, slots=6, max_pages=12, layers=2, heads=2, dim=64, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.shape = (layers, heads, dim)
        self.dtype, self.g = dtype, g
        self.k = torch.empty(layers, pages, page, heads, dim, dtype=dtype, device=DEV).normal_(generator=g)
        self.v = torch.empty_like(self.k).normal_(generator=g)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
        self.table = torch.full((slots, max_pages), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(slots, dtype=torch.int32, device=DEV)
        self.status = torch.zeros(4, dtype=torch.int32, device=DEV)
        self.cache = moe.make_attn_cache(self.k, self.v, self.refs, self.table, self.lens, self.status)
        self.model = Pages(*[t.float().cpu().numpy() for t in (self.k, self.v)],
                           *[t.cpu().numpy().copy() for t in (self.refs, self.table, self.lens)])

    def rows(self, n):
        layers, heads, dim = self.shape
        return [torch.empty(layers, n, heads, dim, dtype=self.dtype, device=DEV).normal_(generator=self.g)
                for _ in range(2)]

    def append(self, counts, slots=None, keep=None, path=None, model=True, behind=0, **call):
        off = np.concatenate([[0], np.cumsum(counts)])
        N, B = int(off[-1]) + behind, len(counts)
        kn, vn = self.rows(N)
        ws = torch.full((moe.attn_cache_append_workspace_bytes(self.cache, B, N),), 0xFF, dtype=torch.uint8, device=DEV)
        moe.attn_cache_append(self.cache, kn, vn, i32(off.tolist()), B, ws, slots=None if slots is None else i32(slots),
                              path=None if path is None else i32(path), n_keep=None if keep is None else i32(keep), **call)
        if model:
            kf, vf = kn.float().cpu().numpy(), vn.float().cpu().numpy()
            jobs = []
            for b in range(B):
                n = counts[b] if keep is None else keep[b]
                pick = [off[b] + (i if path is None else path[b][i]) for i in range(n)]
                jobs.append((b if slots is None else slots[b], kf[:, pick], vf[:, pick]))
            self.model.append(jobs)

    def fork(self, pairs, model=True):
        ws = torch.full((moe.attn_cache_fork_workspace_bytes(self.cache, len(pairs)),), 0xFF, dtype=torch.uint8, device=DEV)
        moe.attn_cache_fork(self.cache, i32([a for a, _ in pairs]), i32([b for _, b in pairs]), len(pairs), ws)
        if model:
            self.model.fork(pairs)

    def trim(self, pairs, model=True):
        moe.attn_cache_trim(self.cache, i32([s for s, _ in pairs]), i32([n for _, n in pairs]), len(pairs))
        if model:
            for s, n in pairs:
                self.model.trim(s, n)

    def check(self, status=0):
        torch.cuda.synchronize()
        assert int(self.status[0]) == status
        self.status.zero_()
        for name in ("refs", "table", "lens"):
            np.testing.assert_array_equal(getattr(self, name).cpu().numpy(), getattr(self.model, name), err_msg=name)
        for name in ("k", "v"):
            np.testing.assert_array_equal(getattr(self, name).float().cpu().numpy(), getattr(self.model, name))


@pytest.mark.parametrize("page,heads,dim,dtype", [(16, 2, 64, torch.bfloat16), (64, 1, 128, torch.float16),
                                                  (32, 3, 256, torch.bfloat16), (128, 8, 64, torch.float16),
                                                  (256, 2, 256, torch.bfloat16)])
def test_a_life_of_a_cache(page, heads, dim, dtype):
    t = Twin(page=page, heads=heads, dim=dim, dtype=dtype, pages=60)
    t.append([page, 1, 0, 2 * page + 3], behind=2)          # exact, one, none, several pages
    t.check()
    t.append([5, page - 1], slots=[3, 1], keep=[2, page - 1], path=[[4, 0] + [0] * page, list(range(page - 1)) + [0] * 3])
    t.check()
    t.fork([(3, 4), (3, 5), (0, 2)])
    t.check()
    t.append([1, 1, 1], slots=[5, 4, 3])                     # everyone behind the fork writes a page of its own
    t.check()
    t.trim([(3, page + 1), (4, 2 * page), (0, 0)])
    t.check()
    t.trim([(5, page + 2)])                                  # inside a page that 3 and 4 share
    t.append([3, 2], slots=[5, 3])                           # both move its rows first
    t.check()
    t.trim([(s, 0) for s in range(6)])
    t.check()
    assert int(t.refs.abs().sum()) == 0 and (t.table == -1).all()


@pytest.mark.parametrize("pages", [37, 61, 2050])
def test_pools_of_odd_sizes_are_used_to_the_last_page(pages):
    t = Twin(pages=pages, slots=2, max_pages=pages, layers=1, heads=1)
    t.append([16 * pages - 5])
    t.trim([(0, 16 * pages - 40)])
    t.append([20], slots=[1])
    t.check()
    t.append([17], slots=[0], model=False)
    t.check(moe.MOE_ERR_OUT_OF_PAGES)
    t.append([3])
    t.check()


def test_random_calls():
    rng = np.random.default_rng(3)
    t = Twin(pages=300, slots=24, max_pages=20, layers=1, heads=1, page=16)
    for _ in range(60):
        lens = t.model.lens
        what = rng.integers(3)
        if what == 0:
            slots = rng.permutation(24)[:rng.integers(1, 25)].tolist()
            t.append([int(min(rng.integers(0, 40), 320 - lens[s])) for s in slots], slots=slots)
        elif what == 1:
            full, empty = np.flatnonzero(lens > 0), np.flatnonzero(lens == 0)
            n = min(len(empty), int(rng.integers(1, 5)))
            if n and len(full):
                t.fork([(int(rng.choice(full)), int(d)) for d in rng.permutation(empty)[:n]])
        else:
            t.trim([(int(s), int(rng.integers(0, lens[s] + 1))) for s in rng.permutation(24)[:rng.integers(1, 12)]])
        if (t.model.refs == 0).sum() < 80:
            t.trim([(int(s), 0) for s in range(24) if lens[s] > 100])
    t.check()


def test_many_sequences_and_a_large_pool():
    t = Twin(pages=20000, slots=1024, max_pages=30, layers=1, heads=1)
    rng = np.random.default_rng(4)
    t.append(rng.integers(0, 200, 1024).tolist())
    t.check()
    slots = rng.permutation(1024).tolist()
    t.append(rng.integers(0, 200, 1024).tolist(), slots=slots)
    t.trim([(s, int(t.model.lens[s]) // 2) for s in slots[:1000]])
    t.check()


def test_the_pool_can_be_used_up_and_no_further():
    t = Twin(pages=4)
    t.append([64])
    t.check()
    t.append([1], slots=[1], model=False)
    t.check(moe.MOE_ERR_OUT_OF_PAGES)
    t.fork([(0, 1)])                   # full pages only: nothing to allocate
    t.check()
    t.trim([(1, 63)])
    t.append([1, 1], slots=[1, 2], model=False)  # one would need a copy, the other a page: neither happens
    t.check(moe.MOE_ERR_OUT_OF_PAGES)
    t.trim([(1, 0)])
    t.trim([(0, 50)])
    t.fork([(0, 3)], model=False)
    t.check(moe.MOE_ERR_OUT_OF_PAGES)
    t.trim([(0, 48)])
    t.append([16], slots=[5])
    t.check()


@pytest.mark.parametrize("bad", ["slot", "twice", "keep", "keep_low", "path", "stride", "room", "offsets", "rows"])
def test_append_device_checks_change_nothing(bad):
    t = Twin(max_pages=3)
    t.append([20, 17])
    t.check()
    args = {"slot": dict(counts=[2, 2], slots=[0, 6]), "twice": dict(counts=[2, 2], slots=[1, 1]),
            "keep": dict(counts=[2, 2], keep=[2, 3]), "keep_low": dict(counts=[2, 2], keep=[-1, 2]),
            "path": dict(counts=[2, 2], keep=[1, 2], path=[[0, 0], [0, 2]]),
            "stride": dict(counts=[5, 2], keep=[3, 1], path=[[0, 1], [0, 1]]),
            "room": dict(counts=[2, 32]), "offsets": dict(counts=[2, 2]), "rows": dict(counts=[2, 2])}[bad]
    if bad in ("offsets", "rows"):
        kn, vn = t.rows(4)
        ws = torch.zeros(moe.attn_cache_append_workspace_bytes(t.cache, 2, 4), dtype=torch.uint8, device=DEV)
        moe.attn_cache_append(t.cache, kn, vn, i32([0, 3, 2] if bad == "offsets" else [0, 2, 5]), 2, ws)
    else:
        t.append(model=False, **args)
    t.check(moe.MOE_ERR_DEVICE_BOUNDS)


@pytest.mark.parametrize("pairs", [[(0, 6)], [(-1, 3)], [(0, 1)], [(0, 3), (1, 3)], [(0, 3), (3, 4)], [(2, 2)]])
def test_fork_device_checks_change_nothing(pairs):
    t = Twin()
    t.append([20, 17])
    t.fork(pairs, model=False)
    t.check(moe.MOE_ERR_DEVICE_BOUNDS)


def test_trim_device_checks_are_per_sequence():
    t = Twin()
    t.append([20, 17, 40])
    t.trim([(0, 21), (1, 3), (9, 0), (2, -1)], model=False)
    t.model.trim(1, 3)
    t.check(moe.MOE_ERR_DEVICE_BOUNDS)
    t.trim([(2, 10), (2, 0)], model=False)  # named twice: the first counts
    t.model.trim(2, 10)
    t.check(moe.MOE_ERR_DEVICE_BOUNDS)


def test_binding_refusals():
    t = Twin()
    kn, vn = t.rows(3)
    ws = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    for bad in (dict(k=kn.float()), dict(k=kn[:1]), dict(off=i32([0, 3]).long()), dict(ws=ws.cpu()), dict(off=i32([0, 1, 3]))):
        a = {**dict(k=kn, off=i32([0, 3]), ws=ws), **bad}
        with pytest.raises(ValueError):
            moe.attn_cache_append(t.cache, a["k"], vn, a["off"], 1, a["ws"])
    with pytest.raises(ValueError):
        moe.attn_cache_trim(t.cache, i32([0]), i32([0, 1]), 1)
    with pytest.raises(ValueError):
        moe.make_attn_cache(t.k, t.v, t.refs[:-1], t.table, t.lens, t.status)
    t.check()


def test_calls_with_nothing_to_do():
    t = Twin()
    t.append([0, 0])
    t.append([3, 2], keep=[0, 0], path=[[0], [0]])
    t.fork([(0, 1)])  # an empty sequence forks into an empty one
    t.trim([(0, 0), (1, 0)])
    t.check()


def test_an_append_replays_from_a_graph():
    t = Twin(layers=3)
    t.append([10, 30])
    t.check()
    kn, vn = t.rows(6)
    off, keep, path = i32([0, 3, 6]), i32([2, 1]), i32([[0, 2], [1, 0]])
    ws = torch.zeros(moe.attn_cache_append_workspace_bytes(t.cache, 2, 6), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            moe.attn_cache_append(t.cache, kn, vn, off, 2, ws, path=path, n_keep=keep)
    torch.cuda.synchronize()
    kf, vf = kn.float().cpu().numpy(), vn.float().cpu().numpy()
    for new_path in ([[0, 2], [1, 0]], [[1, 1], [2, 0]], [[2, 0], [0, 0]]):
        path.copy_(i32(new_path))
        g.replay()
        t.model.append([(0, kf[:, new_path[0]], vf[:, new_path[0]]),
                        (1, kf[:, [3 + new_path[1][0]]], vf[:, [3 + new_path[1][0]]])])
        t.check()


def corrupt(t, slot, block, page):
    t.table[slot, block] = page
    t.model.table[slot, block] = page


@pytest.mark.parametrize("page", [-1, -7, 40, 2 ** 31 - 1])
@pytest.mark.parametrize("block", [0, 1, 70])
def test_a_fork_of_a_table_with_a_bad_entry_changes_nothing(page, block):
    # blocks 0, 1 and 70 are full pages: shared, not copied
    t = Twin(pages=40 if block < 70 else 100, max_pages=90)
    if page == 40:
        page = t.k.shape[1]
    t.append([20, 16 * 71 + 3 if block == 70 else 40])
    t.fork([(0, 4)])
    corrupt(t, 1, block, page)
    t.fork([(0, 2), (1, 3)], model=False)
    t.check(moe.MOE_ERR_DEVICE_BOUNDS)
    t.fork([(1, 3)], model=False)
    t.check(moe.MOE_ERR_DEVICE_BOUNDS)
    t.fork([(0, 2)])
    t.check()


def test_a_fork_of_many_long_sequences():
    # every source's table is gone over by the whole plan, however the entries fall
    t = Twin(pages=3000, slots=400, max_pages=130, layers=1, heads=1)
    lens = [16 * 128 + 5, 0, 16, 1, 16 * 97, 400]
    t.append(lens)
    t.fork([(i % 6, 6 + i) for i in range(390)])
    t.check()
    corrupt(t, 4, 96, 3000)
    t.trim([(s, 0) for s in range(6, 396)])
    t.fork([(i % 6, 6 + i) for i in range(390)], model=False)
    t.check(moe.MOE_ERR_DEVICE_BOUNDS)


@pytest.mark.parametrize("page", [-1, -7, 40, 2 ** 31 - 1])
@pytest.mark.parametrize("block", [1, 2, 140])
def test_a_trim_over_a_bad_entry_leaves_that_sequence_as_it_was(page, block):
    t = Twin(pages=40 if block < 140 else 400, max_pages=150)
    if page == 40:
        page = t.k.shape[1]
    t.append([50, 60, 16 * 143 if block == 140 else 55])
    corrupt(t, 2, block, page)
    t.trim([(0, 5), (2, 3), (1, 0)], model=False)
    t.model.trim(0, 5)
    t.model.trim(1, 0)
    t.check(moe.MOE_ERR_DEVICE_BOUNDS)
    t.trim([(2, 16 * block + 16)])  # behind the bad entry: nothing wrong there
    t.check()


def test_a_trim_of_a_page_that_nobody_holds_leaves_the_sequence_as_it_was():
    t = Twin()
    t.append([50, 40])
    t.refs[t.table[0, 2].long()] = 0
    t.model.refs[t.model.table[0, 2]] = 0
    t.trim([(0, 3), (1, 20)], model=False)
    t.model.trim(1, 20)
    t.check(moe.MOE_ERR_DEVICE_BOUNDS)
