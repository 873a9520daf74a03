"""GPU parity of the tree attention over a paged cache (attn_tree) against the
fp64 oracle.

Tolerance, from the arithmetic.  With u half a step of the type (bf16 2^-8,
fp16 2^-11), o is rounded once: u |o|.  The softmax weights are rounded to the type
for the product with V: at most u sum p|v|, and below fp16's normal range at
most 2^-25 of the largest weight each: 2^-25 sum |v| (bf16: 2^-134, nothing).
Scores are fp32 sums of D products: each is off by at most (D + 2) 2^-24 max
sum |q k| scale =: d, the base-2 exponential and the scores' scaling by 2^-20
relative; a weight's relative error 2 d + 2^-20 enters once through the weight and once
through the sum.  fp32 sums of l terms: l 2^-24 sum p|v|.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle.tree import tree_attention

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import bit_grouped_expert_gb300 as moe  # noqa: E402

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_grouped_expert_gb300 import build
    build.build()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def tree_of(rng, n):
    return [-1] + [int(rng.integers(max(0, i - 9), i)) for i in range(1, n)]


class Case:
    """B sequences over a pool whose unused rows hold NaN, their trees, and the expected output."""

    def __init__(self, seed, lens, trees, Hq=16, Hkv=2, D=256, page=64, dtype="bf16", layers=1, layer=0, gain=1.0,
                 slots=None, extra_pages=3):
        rng = np.random.default_rng(seed)
        t = TYPES[dtype]
        self.lens, self.trees, self.D, self.Hq, self.dtype, self.layer = lens, trees, D, Hq, t, layer
        B, used = len(lens), [-(-L // page) for L in lens]
        P = sum(used) + extra_pages
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)

        def normal(*s):
            return torch.empty(s, dtype=t, device=DEV).normal_(generator=g)

        self.k = torch.full((layers, P, page, Hkv, D), float("nan"), dtype=t, device=DEV)
        self.v = torch.full_like(self.k, float("nan"))
        order = rng.permutation(P)
        self.slots = list(range(B)) if slots is None else slots
        n_slots = max(self.slots) + 1
        table = np.full((n_slots, max(used + [1])), -1)
        slot_lens = np.zeros(n_slots, int)
        refs = np.zeros(P, int)
        self.old = []
        at = 0
        for b in range(B):
            pages = order[at:at + used[b]]
            at += used[b]
            table[self.slots[b], :used[b]] = pages
            slot_lens[self.slots[b]] = lens[b]
            refs[pages] = 1
            k, v = normal(lens[b], Hkv, D), normal(lens[b], Hkv, D)
            self.old.append((k, v))
            idx = torch.from_numpy(pages).to(DEV).repeat_interleave(page)[:lens[b]]
            row = torch.arange(lens[b], device=DEV) % page
            self.k[layer, idx, row] = k
            self.v[layer, idx, row] = v
        self.table, self.slot_lens = i32(table.tolist()), i32(slot_lens.tolist())
        self.refs, self.status = i32(refs.tolist()), torch.zeros(4, dtype=torch.int32, device=DEV)
        counts = [len(p) for p in trees]
        self.off = np.concatenate([[0], np.cumsum(counts)])
        N = int(self.off[-1]) + 2  # two rows behind the last tree
        self.q, self.kn, self.vn = normal(N, Hq, D) * gain, normal(N, Hkv, D), normal(N, Hkv, D)
        self.parent = [p for tree in trees for p in tree] + [-2, -2]
        for i, p in enumerate(self.parent):
            if p == -2:
                self.kn[i] = float("nan")
                self.vn[i] = float("inf")
        self.cache = moe.make_attn_cache(self.k, self.v, self.refs, self.table, self.slot_lens, self.status)
        self.max_nodes = max(counts + [1])
        self.ws = torch.full((moe.attn_tree_workspace_bytes(self.cache, max(B, 1), N, self.max_nodes, Hq),), 0xFF,
                             dtype=torch.uint8, device=DEV)
        self.offsets, self.par = i32(self.off.tolist()), i32(self.parent)
        self.slots_t = None if slots is None else i32(slots)
        self.o = torch.full((N, Hq, D), 7.0, dtype=t, device=DEV)

    def call(self, scale=0.0, stream=None, o=None):
        o = self.o if o is None else o
        moe.attn_tree(self.cache, self.layer, self.q, self.kn, self.vn, self.offsets, self.par, len(self.lens),
                      self.max_nodes, self.ws, o, slots=self.slots_t, scale=scale, stream=stream)
        return o

    def run(self, **kw):
        o = self.call(**kw)
        torch.cuda.synchronize()
        assert self.status.tolist() == [0, 0, 0, 0]
        return o

    def check(self, o, scale=None):
        f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
        assert (o[self.off[-1]:] == 7.0).all(), "rows behind the last tree were written"
        u = torch.finfo(self.dtype).eps / 2
        for b, (L, tree) in enumerate(zip(self.lens, self.trees)):
            lo, hi = self.off[b], self.off[b + 1]
            if lo == hi:
                continue
            ref, wv, av, big = tree_attention(f64(self.q[lo:hi]), f64(self.old[b][0]), f64(self.old[b][1]),
                                              f64(self.kn[lo:hi]), f64(self.vn[lo:hi]), tree, scale)
            d = ((self.D + 2) * 2.0 ** -24 * big)[..., None]
            allow = u * np.abs(ref) + (u + 2 * (2 * d + 2.0 ** -20) + (L + hi - lo) * 2.0 ** -24) * (1 + u) * wv
            if self.dtype == torch.float16:
                allow += 2.0 ** -25 * (av + 1)  # the output's own subnormal step as well
            got = f64(o[lo:hi])
            assert np.isfinite(got).all(), f"tree {b}: non-finite output"
            over = (np.abs(got - ref) - allow).max()
            assert over <= 0, f"tree {b} (len {L}, {hi - lo} nodes): beyond its allowance by {over:.3g}"


SHAPES = [(16, 2, 256, 64, "bf16"), (8, 8, 64, 16, "fp16"), (12, 2, 128, 32, "bf16"), (32, 2, 256, 128, "fp16"),
          (4, 1, 64, 256, "bf16"), (128, 1, 128, 16, "bf16"), (3, 3, 256, 16, "fp16")]


@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", SHAPES)
def test_ragged_batches(Hq, Hkv, D, page, dtype):
    rng = np.random.default_rng(Hq + D)
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1000]
    trees = [tree_of(rng, n) for n in (1, 2, 3, 5, 8, 13, 16, 17, 1, 4, 7, 2, 9)]
    c = Case(1, lens, trees, Hq, Hkv, D, page, dtype)
    c.check(c.run())


@pytest.mark.parametrize("n", [1, 2, 31, 63, 64, 65, 128, 129, 256])
@pytest.mark.parametrize("shape", ["chain", "tree"])
def test_tree_sizes(n, shape):
    tree = list(range(-1, n - 1)) if shape == "chain" else tree_of(np.random.default_rng(n), n)
    c = Case(n, [70, 3], [tree, [-1]], Hq=4, Hkv=2, D=64, page=16)
    c.check(c.run())


def test_one_token_agrees_with_attn_decode():
    L = 3000
    c = Case(3, [L], [[-1]], page=64)
    o = c.run()
    c.check(o)
    k = torch.cat([c.old[0][0], c.kn[:1]]).contiguous()
    v = torch.cat([c.old[0][1], c.vn[:1]]).contiguous()
    ws = torch.zeros(moe.attn_decode_workspace_bytes(L + 1), dtype=torch.uint8, device=DEV)
    ref = torch.empty(16, 256, dtype=torch.bfloat16, device=DEV)
    moe.attn_decode(c.q[0].contiguous(), k, v, L + 1, 16, 2, 256, ws, ref)
    # each is within its allowance of the exact value: at most 2 u |o| + 2 u sum p|v| (u = 2^-8) apart, both below 2 u max|v|
    assert (o[0].float() - ref.float()).abs().max() <= 4 * 2.0 ** -8 * float(v.float().abs().max())


def test_padding_empty_trees_and_empty_sequences():
    trees = [[-1, 0, -2, 1, -2], [], [-2, -2], [-1, 0, 0, -2], [-1]]
    c = Case(4, [100, 50, 40, 0, 0], trees)
    o = c.run()
    c.check(o)
    assert (o[2] == 0).all() and (o[4:7] == 0).all()  # padding rows are zeros


def test_a_row_tile_of_padding_only():
    # 16 nodes a row tile: the second one is padding
    c = Case(22, [150], [tree_of(np.random.default_rng(4), 16) + [-2] * 16 + [15] * 8])
    o = c.run()
    c.check(o)
    assert (o[16:32] == 0).all()


def test_no_nodes_at_all():
    c = Case(23, [150, 0], [[], []])
    c.check(c.run())


def test_many_kv_heads():
    c = Case(24, [70, 5], [[-1, 0], [-1]], Hq=128, Hkv=64, D=64, page=32)
    c.check(c.run())


def test_trees_of_uneven_sizes_and_long_caches():
    # teams of row tiles that some trees leave empty, and the same work cut alone
    rng = np.random.default_rng(5)
    c = Case(25, [4000, 3500, 3000, 3900], [tree_of(rng, n) for n in (60, 50, 64, 33)], page=128)
    c.check(c.run())
    c = Case(26, [4000, 3500, 3000, 3900], [tree_of(rng, n) for n in (64, 1, 2, 1)], page=128)
    c.check(c.run())


def test_several_roots_see_only_their_own_tree():
    c = Case(5, [20], [[-1, -1, 0, 1, -1, 4]], D=128, Hq=8)
    c.check(c.run())


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_other_branches_cannot_change_a_row(bad, dtype):
    # node 1 and its children hold non-finite K and V: only rows that see node 1 may show it
    tree = [-1, 0, 0, 1, 2, 1, 4]
    c = Case(6, [90, 33], [tree, [-1, 0]], dtype=dtype, D=128, Hq=16)
    good = c.run().clone()
    for i in (1, 3, 5):
        c.vn[i, :, ::3] = bad
        c.kn[i, 1] = bad
    o = c.run()
    assert torch.equal(o[[0, 2, 4, 6, 7, 8]], good[[0, 2, 4, 6, 7, 8]])
    assert not torch.isfinite(o[[1, 3, 5]].float()).all(-1).any()


def test_infinite_values_reach_the_rows_that_see_them():
    c = Case(7, [30], [[-1, 0, 0]])
    c.vn[1, :, 5] = float("inf")
    o = c.run().float()
    assert torch.isinf(o[1, :, 5]).all() and (o[1, :, 5] > 0).all()
    keep = [d for d in range(256) if d != 5]
    assert torch.isfinite(o[1][:, keep]).all() and torch.isfinite(o[[0, 2]]).all()


@pytest.mark.parametrize("scale,gain", [(0.0, 30.0), (1.0, 1.0), (1e-3, 1.0), (0.05, 0.0)])
def test_peaked_and_flat_scores(scale, gain):
    c = Case(8, [700, 64], [tree_of(np.random.default_rng(0), 9), [-1]], gain=gain)
    c.check(c.run(scale=scale), scale or None)


def test_rising_and_falling_scores():
    # keys grow along the cache, so the running maximum moves at every tile (and never, reversed)
    c = Case(9, [2000, 2000], [[-1, 0, 1], [-1]])
    for b, ramp in ((0, torch.linspace(0, 4, 2000, device=DEV)), (1, torch.linspace(4, 0, 2000, device=DEV))):
        k = (c.old[b][0].float() * 0.05 + ramp[:, None, None] * torch.sign(c.q[c.off[b], 0].float())).to(c.dtype)
        c.old[b] = (k, c.old[b][1])
        pages = c.table[b].long().repeat_interleave(64)[:2000]
        c.k[0, pages, torch.arange(2000, device=DEV) % 64] = k
    c.check(c.run())


def test_slots_layers_and_a_sequence_read_twice():
    c = Case(10, [77, 130], [[-1, 0], [-1, 0, 1]], layers=3, layer=2, slots=[4, 1], page=32)
    o = c.run()
    c.check(o)
    # both trees over slot 1
    c2 = Case(10, [77, 130], [[-1, 0], [-1, 0, 1]], layers=3, layer=2, slots=[4, 1], page=32)
    c2.slots_t = i32([1, 1])
    c2.old[0], c2.lens = c2.old[1], [130, 130]
    c2.check(c2.run())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_a_long_cache_with_a_wide_tree(dtype):
    c = Case(11, [40000], [tree_of(np.random.default_rng(2), 40)], Hq=16, Hkv=2, D=256, page=128, dtype=dtype)
    c.check(c.run())


def test_many_sequences():
    rng = np.random.default_rng(12)
    lens = [int(x) for x in rng.integers(0, 90, 1000)]
    trees = [tree_of(rng, int(x)) for x in rng.integers(1, 4, 1000)]
    c = Case(12, lens, trees, Hq=2, Hkv=1, D=64, page=16)
    c.check(c.run())


def test_offsets_beyond_31_bits():
    # 4 layers x 17500 pages x 64 x 2 x 256 = 2.29e9 values: the last layer starts beyond 2^31 - 1
    L, layers, P = 500, 4, 17500
    c = Case(13, [L], [[-1, 0, 1]])
    k = torch.empty(layers, P, 64, 2, 256, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    pages = torch.arange(P - 8, P, device=DEV)
    k[3, pages] = c.k[0, c.table[0].long()]
    v[3, pages] = c.v[0, c.table[0].long()]
    c.table[0] = pages.to(torch.int32)
    c.cache = moe.make_attn_cache(k, v, torch.zeros(P, dtype=torch.int32, device=DEV), c.table, c.slot_lens, c.status)
    c.layer = 3
    c.check(c.run())


def test_calls_repeat_exactly_and_replay_from_a_graph():
    c = Case(14, [5000, 130, 0], [tree_of(np.random.default_rng(3), 20), [-1, 0], [-1]])
    first = c.run().clone()
    assert torch.equal(c.run(), first)
    c.o.fill_(7.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.call()
        g.replay()
    s.synchronize()
    assert torch.equal(c.o, first)
    # the graph reads lengths and tables anew
    c.slot_lens[1] = 64
    c.old[1] = (c.old[1][0][:64], c.old[1][1][:64])
    c.lens[1] = 64
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    c.check(c.o)


def test_two_streams_with_a_workspace_each():
    cs = [Case(15 + i, [3000 + 500 * i], [tree_of(np.random.default_rng(i), 12)]) for i in range(2)]
    want = [c.run().clone() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(cs, streams):
            c.call(stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cs, want):
        assert torch.equal(c.o, w)


@pytest.mark.parametrize("what", ["slot", "slot_low", "offset", "order", "max_nodes", "parent", "parent_self", "padded_parent",
                                  "len", "page"])
def test_device_checks(what):
    c = Case(20, [100, 70], [[-1, 0, 1], [-1, 0]])
    c.slots_t = i32([0, 1])
    if what == "slot":
        c.slots_t = i32([0, 2])
    elif what == "slot_low":
        c.slots_t = i32([-1, 1])
    elif what == "offset":
        c.offsets = i32([0, 3, 8])
    elif what == "order":
        c.offsets = i32([0, 5, 3])
    elif what == "max_nodes":
        c.max_nodes = 2
    elif what == "parent":
        c.par[1] = 2
    elif what == "parent_self":
        c.par[1] = -3
    elif what == "padded_parent":
        c.par[1] = -2  # and node 2 is its child
    elif what == "len":
        c.slot_lens[0] = 129
    elif what == "page":
        c.table[0, 1] = c.k.shape[1]
    c.call()
    torch.cuda.synchronize()
    assert int(c.status[0]) == moe.MOE_ERR_DEVICE_BOUNDS
    assert (c.o[5:] == 7.0).all()


def test_binding_refusals():
    c = Case(21, [10], [[-1, 0]])
    with pytest.raises(ValueError, match="q"):
        moe.attn_tree(c.cache, 0, c.q.float(), c.kn, c.vn, c.offsets, c.par, 1, 2, c.ws, c.o)
    with pytest.raises(ValueError, match="not contiguous"):
        moe.attn_tree(c.cache, 0, c.q, c.kn.transpose(0, 1).contiguous().transpose(0, 1), c.vn, c.offsets, c.par, 1, 2,
                      c.ws, c.o)
    with pytest.raises(ValueError, match="offsets"):
        moe.attn_tree(c.cache, 0, c.q, c.kn, c.vn, c.offsets.cpu(), c.par, 1, 2, c.ws, c.o)
    with pytest.raises(ValueError, match="ws"):
        moe.attn_tree(c.cache, 0, c.q, c.kn, c.vn, c.offsets, c.par, 1, 2, c.ws.cpu(), c.o)
    with pytest.raises(moe.MoeError, match="workspace too small"):
        moe.attn_tree(c.cache, 0, c.q, c.kn, c.vn, c.offsets, c.par, 1, 2, c.ws[:64], c.o)
    with pytest.raises(ValueError, match="parent"):
        moe.attn_tree(c.cache, 0, c.q, c.kn, c.vn, c.offsets, c.par[:2], 1, 2, c.ws, c.o)


SPLITS = [([0], "whole"), ([64], "two CTAs"), ([3000], "many CTAs"), ([100] * 200, "more units than CTAs"),
          ([20000, 5, 700], "uneven")]


@pytest.mark.parametrize("lens", [s[0] for s in SPLITS], ids=[s[1] for s in SPLITS])
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "fp16"), (256, "bf16")])
def test_a_query_that_is_not_a_number_gives_none_however_the_work_is_cut(lens, D, dtype):
    c = Case(27, lens, [[-1, 0]] * len(lens), Hq=8, D=D, dtype=dtype)
    good = c.run().clone()
    rows = [(0, 3), (1, 6)]  # (node, head)
    for i, h in rows:
        c.q[i, h, D // 2] = float("nan")
    o = c.run()
    hit = torch.zeros(o.shape[:2], dtype=torch.bool, device=DEV)
    for i, h in rows:
        hit[i, h] = True
    assert torch.isnan(o[hit].float()).all()
    assert torch.equal(o[~hit], good[~hit])


@pytest.mark.parametrize("L,lo,hi", [(64, 0, 64), (300, 128, 256), (3000, 1024, 1280), (3000, 0, 3000), (3000, 1500, 1501),
                                     (20000, 4096, 9000)])
@pytest.mark.parametrize("D", [64, 256])
def test_cached_keys_that_are_not_numbers_show_however_the_work_is_cut(L, lo, hi, D):
    # a whole CTA's part of them, several, all, or one position
    c = Case(28, [L, 130], [[-1, 0], [-1]], Hq=8, Hkv=2, D=D)
    good = c.run().clone()
    pos = torch.arange(lo, hi, device=DEV)
    c.k[0, c.table[0].long()[pos // 64], pos % 64, 1] = float("nan")
    o = c.run()
    assert torch.isnan(o[:2, 4:].float()).all()
    assert torch.equal(o[:2, :4], good[:2, :4]) and torch.equal(o[2:], good[2:])


@pytest.mark.parametrize("L", [64, 3000])
def test_cached_values_that_are_not_numbers_show_in_their_columns(L):
    c = Case(29, [L], [[-1, 0]], Hq=8, Hkv=2, D=128)
    good = c.run().clone()
    c.v[0, int(c.table[0, 0]), 7, 0, 5] = float("nan")
    o = c.run()
    assert torch.isnan(o[:2, :4, 5].float()).all()
    o[:2, :4, 5] = good[:2, :4, 5]
    assert torch.equal(o, good)


@pytest.mark.parametrize("Hq,Hkv,D,dtype,n", [(5, 1, 64, "bf16", 40), (14, 2, 128, "fp16", 19), (127, 1, 64, "bf16", 3),
                                              (66, 2, 256, "bf16", 9), (128, 1, 64, "fp16", 256)])
def test_groups_of_odd_sizes_and_the_most_row_tiles(Hq, Hkv, D, dtype, n):
    # the last: 256 row tiles of one node, more than a team can have CTAs
    c = Case(32, [200, 0], [tree_of(np.random.default_rng(n), n), [-1]], Hq=Hq, Hkv=Hkv, D=D, page=32, dtype=dtype)
    c.check(c.run())
