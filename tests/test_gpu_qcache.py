"""GPU parity of the 8-bit paged cache (attn_qcache_append, _fork, _trim,
_attend) against the fp64 oracle.

Appending without rotation is exact: a value of the rows' type divided by a power of
two, rounded once; scales, codes, tables and holders are compared for equality.
With rotation the row is off by (|x| + |y|) (2^-20 + |p| 2^-49) before its code is
taken (tests/test_gpu_rotary.py): the code is then within half a step, of it or
of its neighbour, plus that.

Attention, with u half a step of q's type (bf16 2^-8, fp16 2^-11 and at least 2^-25).  o is
rounded once: u |o|.  q is cut into e4m3 parts that keep all of its bits but for 2^-10 2^e, where
2^e >= its row's largest / 448; scores are fp32 sums of 3 D products at most.  So a score is off by
d = scale (D 2^-22 sum |q k| + 2^-10 2^e sum |k|), and a weight, with its exponential, by
e^d (1 + 2^-20) - 1, which enters once through the weight and once through the sum.  The weights are
rounded to fp16, 2^-11, and cut into three e5m2 parts, 2^-11 or 2^-23 of the largest weight times the
largest scale of V: 2^-10 together.
fp32 sums of 3 l terms.  Together
  u |o| + sum p|v| (2^-10 + 2 (e^d (1 + 2^-20) - 1) + l 2^-21) + 2^-22 max p max s sum |code|.
Most roundings fall on either side: for zero-mean values the norm of the error is that of
independent errors uniform within u and 2^-10 of o, over sqrt 3 each: below
0.6 sqrt(u^2 + 2^-20) of o's norm.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle.qcache import QPages, attend, nearest, scale_of
from oracle.rotary import rates, rotate

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import bit_grouped_expert_gb300 as moe  # noqa: E402

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_grouped_expert_gb300 import build
    build.build()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def f64(t):
    return t.float().double().cpu().numpy()


class Twin:
    """A cache on the GPU and the oracle's copy of it; check() holds one against the other."""

    def __init__(self, page=16, heads=2, dim=64, dtype="bf16", pages=40, slots=6, max_pages=12, layers=2, seed=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.shape, self.dtype, self.g = (layers, heads, dim), TYPES[dtype], g
        self.k, self.v = (self.normal(layers, pages, page, heads, dim).float().mul_(50).to(F8) for _ in "kv")
        self.ks, self.vs = (torch.full((layers, pages, heads), 4.0, device=DEV) for _ in "kv")  # left from before
        self.refs, self.lens = i32([0] * pages), i32([0] * slots)
        self.table, self.status = torch.full((slots, max_pages), -1, dtype=torch.int32, device=DEV), i32([0] * 4)
        self.cache = moe.make_attn_qcache(self.k, self.v, self.ks, self.vs, self.refs, self.table, self.lens, self.status)
        self.model = QPages(f64(self.k), f64(self.v), f64(self.ks), f64(self.vs),
                            *[t.cpu().numpy().copy() for t in (self.refs, self.table, self.lens)])

    def normal(self, *s):
        return torch.empty(s, dtype=self.dtype, device=DEV).normal_(generator=self.g)

    def append(self, counts, slots=None, keep=None, path=None, gain=1.0, model=True, rows=None, behind=0):
        layers, heads, dim = self.shape
        off = np.concatenate([[0], np.cumsum(counts)])
        N, B = int(off[-1]) + behind, len(counts)
        kn, vn = rows or [(self.normal(layers, N, heads, dim) * gain).contiguous() for _ in "kv"]
        ws = torch.full((moe.attn_qcache_append_workspace_bytes(self.cache, B, N),), 0xFF, dtype=torch.uint8, device=DEV)
        opt = {n: None if v is None else i32(v) for n, v in (("slots", slots), ("n_keep", keep), ("path", path))}
        moe.attn_qcache_append(self.cache, None, kn, vn, i32(off.tolist()), B, ws, **opt)
        if model:
            kf, vf = f64(kn), f64(vn)
            jobs = []
            for b in range(B):
                n = counts[b] if keep is None else keep[b]
                pick = [off[b] + (i if path is None else path[b][i]) for i in range(n)]
                jobs.append((b if slots is None else slots[b], kf[:, pick], vf[:, pick]))
            self.model.append(jobs)

    def fork(self, pairs, model=True):
        ws = torch.full((moe.attn_qcache_fork_workspace_bytes(self.cache, len(pairs)),), 0xFF, dtype=torch.uint8, device=DEV)
        moe.attn_qcache_fork(self.cache, i32([a for a, _ in pairs]), i32([b for _, b in pairs]), len(pairs), ws)
        if model:
            self.model.fork(pairs)

    def trim(self, pairs):
        moe.attn_qcache_trim(self.cache, i32([s for s, _ in pairs]), i32([n for _, n in pairs]), len(pairs))
        for s, n in pairs:
            self.model.trim(s, n)

    def check(self, status=0):
        torch.cuda.synchronize()
        assert int(self.status[0]) == status
        self.status.zero_()
        for name in ("refs", "table", "lens"):
            np.testing.assert_array_equal(getattr(self, name).cpu().numpy(), getattr(self.model, name), err_msg=name)
        for name in ("ks", "vs", "k", "v"):
            np.testing.assert_array_equal(f64(getattr(self, name)), getattr(self.model, name), err_msg=name)


@pytest.mark.parametrize("page,heads,dim,dtype", [(16, 2, 64, "bf16"), (64, 1, 128, "fp16"), (32, 3, 256, "bf16"),
                                                  (128, 8, 64, "fp16"), (256, 2, 256, "bf16"), (16, 1, 64, "fp16")])
def test_a_life_of_a_cache(page, heads, dim, dtype):
    t = Twin(page, heads, dim, dtype, pages=60)
    t.append([page, 1, 0, 2 * page + 3], behind=2)
    t.check()
    t.append([5, page - 1], slots=[3, 1], keep=[2, page - 1], path=[[4, 0] + [0] * page, list(range(page - 1)) + [0] * 3],
             gain=5.0)                                        # scales grow: earlier rows are rounded again
    t.check()
    t.fork([(3, 4), (3, 5), (0, 2)])
    t.check()
    t.append([1, 1, 1], slots=[5, 4, 3], gain=40.0)           # pages of their own, and larger scales
    t.check()
    t.append([2, 2], slots=[5, 3], gain=0.001)                # scales stay
    t.check()
    t.trim([(3, page + 1), (4, 2 * page), (0, 0)])
    t.check()
    t.trim([(5, page + 2)])
    t.append([3, 2, 4], slots=[5, 3, 4], gain=100.0)
    t.check()
    t.trim([(s, 0) for s in range(6)])
    t.append([3], gain=2.0 ** -7)                             # a page begun anew: nothing left of its scale
    t.check()


def test_random_calls():
    rng = np.random.default_rng(3)
    t = Twin(pages=300, slots=24, max_pages=20, layers=2, heads=3, page=16)
    for _ in range(50):
        lens = t.model.lens
        what = rng.integers(3)
        if what == 0:
            slots = rng.permutation(24)[:rng.integers(1, 25)].tolist()
            t.append([int(min(rng.integers(0, 40), 320 - lens[s])) for s in slots], slots=slots,
                     gain=float(2.0 ** rng.integers(-3, 4)))
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


def test_many_sequences():
    t = Twin(pages=4000, slots=1024, max_pages=12, layers=1, heads=1)
    rng = np.random.default_rng(4)
    t.append(rng.integers(0, 40, 1024).tolist())
    t.append(rng.integers(0, 3, 1024).tolist(), slots=rng.permutation(1024).tolist(), gain=3.0)
    t.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_the_smallest_and_largest_values(dtype):
    t = Twin(dtype=dtype, layers=1, heads=1)
    top = torch.finfo(t.dtype).max
    x = torch.zeros(1, 40, 1, 64, dtype=t.dtype, device=DEV)
    x[0, 0, 0, :4] = torch.tensor([448.0, -448.0, 449.0, 1.0])      # 448 fits exactly, the next value does not
    x[0, 16, 0, 3], x[0, 17, 0, 5] = top, -top / 2
    x[0, 32, 0, 1] = torch.finfo(t.dtype).tiny
    t.append([40], rows=[x, (x * 0.5).contiguous()])
    t.append([3], slots=[1], rows=[torch.zeros_like(x[:, :3]), torch.full_like(x[:, :3], 448.0)])  # a page of zeros
    t.check()
    t.append([1, 1], slots=[0, 1], rows=[x[:, 16:18].contiguous(), x[:, 16:18].contiguous()])
    t.check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite_become_nan_alone(bad):
    t = Twin()
    kn, vn = t.normal(2, 20, 2, 64), t.normal(2, 20, 2, 64)
    kn[0, 3, 1, 5], vn[1, 18, 0, 63], vn[0, 7] = bad, bad, bad
    t.append([20], rows=[kn, vn])
    t.check()
    t.append([2], gain=100.0)
    t.check()


def test_ties_go_to_the_even_code():
    t = Twin(layers=1, heads=1, dtype="fp16")
    x = torch.zeros(1, 16, 1, 64, dtype=torch.float16, device=DEV)
    x[0, 0, 0, 0] = 448.0
    x[0, 1, 0] = torch.arange(64) + 17.0           # steps of 2: every second one lies half way
    x[0, 2, 0] = (torch.arange(64) + 0.5) * 2.0 ** -9
    t.append([16], rows=[x, (-x).contiguous()])
    t.check()


@pytest.mark.parametrize("page,dim,dtype,rdim,inter", [(16, 64, "bf16", 64, True), (64, 256, "fp16", 64, False),
                                                       (256, 128, "bf16", 128, False)])
def test_rotation_on_the_way(page, dim, dtype, rdim, inter):
    t = Twin(page, 2, dim, dtype, layers=2, max_pages=20)
    kw = dict(base=1e6, stretch=8.0, low_turns=1.0, high_turns=32.0, original_len=512)
    rot, w = moe.make_rotary(rdim, interleaved=inter, factor=1.1, **kw), rates(rdim, **kw)
    held = {0: np.zeros((2, 0, 2, dim)), 1: np.zeros((2, 0, 2, dim))}
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)
    for counts in ([page + 5, 3], [1, 2 * page]):
        N = sum(counts)
        kn, vn = t.normal(2, N, 2, dim), t.normal(2, N, 2, dim)
        moe.attn_qcache_append(t.cache, rot, kn, vn, i32([0, counts[0], N]), 2, ws)
        for s, x in ((0, f64(kn)[:, :counts[0]]), (1, f64(kn)[:, counts[0]:])):
            L = held[s].shape[1]
            pos = list(range(L, L + x.shape[1]))
            held[s] = np.concatenate([held[s], np.stack([rotate(x[l], pos, w, inter, 1.1) for l in range(2)])], 1)
    assert int(t.status[0]) == 0
    table, codes, scales = t.table.cpu().numpy(), f64(t.k), f64(t.ks)
    for s in (0, 1):
        for p in range(held[s].shape[1]):
            x, page_no = held[s][:, p], table[s, p // page]
            sc = scales[:, page_no][:, :, None]
            got = codes[:, page_no, p % page] * sc
            # half a step, once more where the page's scale grew; the rotation's own error moves it further
            step = np.maximum(np.abs(x) * 2.0 ** -4, sc * 2.0 ** -10)
            grown = sc * 2.0 ** -10 * (p % page < 5)
            assert (np.abs(got - x) <= step * (1 + 2.0 ** -3) + grown + 20 * 2.0 ** -20).all()
        # every page's scale: the least that holds its rows
        for b in range(-(-held[s].shape[1] // page)):
            x = np.abs(held[s][:, b * page:(b + 1) * page]).max((1, 3))
            want = np.vectorize(scale_of)(x)
            np.testing.assert_array_equal(scales[:, table[s, b]], want)


# Few rows for each sequence, each with values in its fastest pairs only, whose largest turned value hangs on the
# position: the scale is that of the rows that are there (a warp takes 2, 4 or 8 rows at a time).
@pytest.mark.parametrize("dim,rdim,inter", [(64, 64, False), (64, 48, True), (128, 32, False), (256, 64, True), (256, 256, False)])
@pytest.mark.parametrize("n", [1, 3, 9])
def test_scales_of_few_turned_rows(dim, rdim, inter, n):
    B, page = 60, 16
    t = Twin(page, 2, dim, "bf16", pages=100, slots=B, max_pages=1, layers=2, seed=n)
    rot, w = moe.make_rotary(rdim, base=100.0, interleaved=inter), rates(rdim, base=100.0)
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)
    for first in (0, n % 5):
        if first:  # rows before these, small ones
            small = torch.full((2, B * first, 2, dim), 2.0 ** -20, dtype=torch.bfloat16, device=DEV)
            moe.attn_qcache_append(t.cache, rot, small, small, i32([first * b for b in range(B + 1)]), B, ws)
        kn = t.normal(2, B * n, 2, dim)
        pairs = torch.arange(dim, device=DEV)
        fast = pairs // 2 < 2 if inter else pairs % (rdim // 2) < 2
        kn = (kn * (fast & (pairs < rdim))).contiguous()
        before = int(t.lens[0])
        moe.attn_qcache_append(t.cache, rot, kn, kn, i32([n * b for b in range(B + 1)]), B, ws)
        x = f64(kn).reshape(2, B, n, 2, dim)
        pos = range(before, before + n)
        turned = np.stack([[rotate(x[l, b], pos, w, inter) for l in range(2)] for b in range(B)])
        most, ks = np.abs(turned).max((2, 4)), f64(t.ks)[:, t.table.cpu().numpy()[:, 0]].transpose(1, 0, 2)
        want = np.vectorize(scale_of)(most)
        clear = np.abs(most / (448 * want) - 1) > 2.0 ** -12
        clear &= np.abs(most / (224 * want) - 1) > 2.0 ** -12
        assert clear.sum() > 200 and int(t.status[0]) == 0
        assert (ks[clear] == want[clear]).all(), np.argwhere(clear & (ks != want))[:5]
        moe.attn_qcache_trim(t.cache, None, i32([0] * B), B)


@pytest.mark.parametrize("heads,dim,layers,page", [(256, 64, 3, 16), (100, 128, 2, 32), (3, 256, 7, 256)])
def test_many_heads_and_layers(heads, dim, layers, page):
    t = Twin(page, heads, dim, "bf16", pages=8, slots=2, max_pages=3, layers=layers)
    t.append([page + 3, 5])
    t.append([1, 9], gain=6.0)
    t.check()


def test_appends_replay_from_a_graph_with_attention_behind():
    # one graph of an append and the attention over it: the lengths are the device's, so every replay goes on
    t = Twin(16, 2, 128, "bf16", pages=40, slots=2, max_pages=12, layers=1)
    t.append([30, 5])
    kn, vn, q = t.normal(1, 3, 2, 128), t.normal(1, 3, 2, 128), t.normal(3, 8, 128)
    o, off = torch.zeros_like(q), i32([0, 2, 3])
    ws = torch.zeros(max(moe.attn_qcache_append_workspace_bytes(t.cache, 2, 3),
                         moe.attn_qcache_attend_workspace_bytes(t.cache, 2, 3, 2, 8)), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            moe.attn_qcache_append(t.cache, None, kn, vn, off, 2, ws)
            moe.attn_qcache_attend(t.cache, 0, q, off, 2, 2, ws, o)
    torch.cuda.synchronize()
    for k in range(4):
        kn.mul_(1.7)
        g.replay()
        kf, vf = f64(kn), f64(vn)
        t.model.append([(0, kf[:, :2], vf[:, :2]), (1, kf[:, 2:], vf[:, 2:])])
        t.check()
        for slot, lo, n in ((0, 0, 2), (1, 2, 1)):
            ref, mass, _ = attend(f64(q[lo:lo + n]), *t.model.values(slot))
            assert (np.abs(f64(o[lo:lo + n]) - ref) <= mass * 2.0 ** -6 + 2.0 ** -8).all()


def test_append_and_attend_without_tables_of_their_own_size():
    t = Twin(max_pages=3)
    t.append([20, 17])
    t.check()
    t.append([2, 32], model=False)
    t.check(moe.MOE_ERR_DEVICE_BOUNDS)
    t.append([2, 2], slots=[1, 1], model=False)
    t.check(moe.MOE_ERR_DEVICE_BOUNDS)
    t.fork([(0, 1)], model=False)
    t.check(moe.MOE_ERR_DEVICE_BOUNDS)
    small = Twin(pages=2)
    small.append([20])
    small.append([1], slots=[1], model=False)
    small.check(moe.MOE_ERR_OUT_OF_PAGES)


# ------------------------------------------------------------------ attention

class Case:
    """B sequences over a pool whose unused rows hold NaN, and the expected output of their last rows."""

    def __init__(self, seed, lens, counts, Hq=16, Hkv=2, D=256, page=64, dtype="bf16", layers=1, layer=0, slots=None,
                 gain=1.0, pow2=True, behind=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.t = t = TYPES[dtype]
        self.lens, self.counts, self.Hq, self.D, self.layer, self.dtype = lens, counts, Hq, D, layer, dtype
        self.slots = list(range(len(lens))) if slots is None else slots
        n_slots = max(self.slots) + 1
        of = {s: L for s, L in zip(self.slots, lens)}
        used = {s: -(-L // page) for s, L in of.items()}
        P = sum(used.values()) + 3
        order = rng.permutation(P)
        nan = torch.full((layers, P, page, Hkv, D), 0x7F, dtype=torch.uint8, device=DEV)
        self.k, self.v = nan.clone().view(F8), nan.view(F8)
        self.ks, self.vs = (torch.full((layers, P, Hkv), float("nan"), device=DEV) for _ in "kv")
        table, slot_lens, refs = np.full((n_slots, max(list(used.values()) + [1])), -1), np.zeros(n_slots, int), np.zeros(P, int)
        self.old, at = {}, 0
        for s, L in of.items():
            pages = order[at:at + used[s]]
            at += used[s]
            table[s, :used[s]], slot_lens[s], refs[pages] = pages, L, 1
            both = []
            for pool, scales in ((self.k, self.ks), (self.v, self.vs)):
                codes = torch.empty(L, Hkv, D, device=DEV).normal_(generator=g).mul_(100).clamp_(-448, 448).to(F8)
                sc = torch.from_numpy(2.0 ** rng.integers(-8, -5, (used[s], Hkv)) * (1 if pow2 else
                                                                                    rng.uniform(0.5, 1.5, (used[s], Hkv))))
                sc = sc.float().to(DEV)
                i = torch.arange(L, device=DEV)
                p = torch.from_numpy(pages).to(DEV)
                pool.view(torch.uint8)[layer, p[i // page], i % page] = codes.view(torch.uint8)
                scales[layer, p] = sc
                both.append((f64(codes), sc.double()[i // page].cpu().numpy()))
            self.old[s] = both
        self.refs, self.table, self.slot_lens, self.status = i32(refs.tolist()), i32(table.tolist()), i32(slot_lens.tolist()), i32([0])
        self.off = np.concatenate([[0], np.cumsum(counts)])
        N = int(self.off[-1]) + behind
        self.q = torch.empty(N, Hq, D, dtype=t, device=DEV).normal_(generator=g).mul_(gain)
        self.max_rows = max(counts + [1])
        self.cache = moe.make_attn_qcache(self.k, self.v, self.ks, self.vs, self.refs, self.table, self.slot_lens, self.status)
        self.ws = torch.full((moe.attn_qcache_attend_workspace_bytes(self.cache, len(lens), max(N, 1), self.max_rows, Hq),),
                             0xFF, dtype=torch.uint8, device=DEV)
        self.o = torch.full((N, Hq, D), 7.0, dtype=t, device=DEV)

    def run(self, scale=0.0, **kw):
        slots = None if self.slots == list(range(len(self.slots))) else i32(self.slots)
        moe.attn_qcache_attend(self.cache, self.layer, self.q, i32(self.off.tolist()), len(self.lens), self.max_rows, self.ws,
                               self.o, slots=slots, scale=scale, **kw)
        return self.o

    def check(self, scale=0.0, status=0, norm=True):
        torch.cuda.synchronize()
        assert int(self.status[0]) == status
        got, u = f64(self.o), {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[self.dtype]
        G = self.Hq // self.k.shape[3]
        sc = scale or self.D ** -0.5
        err2 = ref2 = 0.0
        for b, s in enumerate(self.slots):
            lo, n, L = int(self.off[b]), self.counts[b], self.lens[b]
            if n == 0:
                continue
            q = f64(self.q[lo:lo + n])
            (kc, ks), (vc, vs) = self.old[s]
            k, v = kc * ks[..., None], vc * vs[..., None]
            o, mass, most = attend(q, k, v, sc)
            if L == 0:
                assert (got[lo:lo + n] == 0).all()
                continue
            unit = np.vectorize(scale_of)(np.abs(q).max(-1))                       # 2^e of a row
            ksum = np.repeat(np.abs(k).sum(-1).max(0), G)
            d = sc * 2.0 ** -10 * unit * ksum + most * self.D * 2.0 ** -22
            top = np.repeat(vs.max(0), G)[:, None] * np.repeat(np.abs(vc).sum(0), G, 0)
            lim = u * np.abs(o) + 2.0 ** -25 + mass * (2.0 ** -10 + 2 * (np.exp(d) * (1 + 2.0 ** -20) - 1)[..., None] +
                                                       L * 2.0 ** -21) + 2.0 ** -22 * top
            e = np.abs(got[lo:lo + n] - o)
            assert (e <= lim).all(), (b, float((e / lim).max()))
            err2, ref2 = err2 + (e ** 2).sum(), ref2 + (o ** 2).sum()
        assert (got[int(self.off[-1]):] == 7.0).all()                                # rows of no sequence
        if norm and ref2:
            assert err2 ** 0.5 <= 0.6 * (u * u + 2.0 ** -20) ** 0.5 * ref2 ** 0.5, (err2 / ref2) ** 0.5


SHAPES = [(16, 2, 256, 64, "bf16"), (16, 2, 256, 128, "fp16"), (32, 8, 128, 16, "fp16"), (8, 8, 64, 32, "bf16"),
          (6, 1, 64, 256, "bf16"), (5, 1, 128, 64, "fp16"), (4, 4, 256, 256, "bf16"), (24, 1, 256, 16, "bf16")]


@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", SHAPES)
def test_one_token_each(Hq, Hkv, D, page, dtype):
    c = Case(1, [1, 2, 127, 128, 129, 700, 1500], [1] * 7, Hq, Hkv, D, page, dtype)
    c.run()
    c.check()


@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", SHAPES)
def test_uneven_chunks(Hq, Hkv, D, page, dtype):
    c = Case(2, [40, 300, 513, 64, 1], [40, 17, 129, 0, 1], Hq, Hkv, D, page, dtype, behind=3)
    c.run()
    c.check()


def test_scales_that_are_not_powers_of_two():
    c = Case(3, [900, 33], [3, 2], pow2=False)
    c.run()
    c.check()


@pytest.mark.parametrize("L", [1, 15, 16, 17, 127, 128, 129, 255, 257, 40000])
def test_lengths(L):
    c = Case(L, [L], [1])
    c.run()
    c.check()


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 33, 200])
def test_row_counts(n):
    c = Case(n, [200], [n])
    c.run()
    c.check()


def test_more_rows_than_the_cache_holds_and_empty_sequences():
    c = Case(4, [5, 0, 0, 130], [9, 3, 0, 131])
    c.run()
    c.check()


@pytest.mark.parametrize("Hq,Hkv", [(128, 1), (127, 1), (7, 7), (30, 2)])
def test_groups_of_odd_sizes(Hq, Hkv):
    c = Case(5, [150, 60], [3, 60], Hq, Hkv, 64)
    c.run()
    c.check()


def test_many_kv_heads():
    c = Case(6, [77], [2], 256, 256, 64)
    c.run()
    c.check()


@pytest.mark.parametrize("scale,gain", [(0.0, 20.0), (1.0, 0.3), (1e-3, 1.0), (0.05, 0.0), (0.0, 1e-30)])
def test_peaked_and_flat_scores(scale, gain):
    c = Case(7, [1000, 3], [2, 3], gain=gain)
    c.run(scale)
    c.check(scale, norm=False)


def test_rising_and_falling_scores_and_scales():
    # the running maximum and the largest scale of V change from tile to tile
    for up in (1, -1):
        c = Case(8, [2000], [1], 8, 1, 128, 16)
        order = c.table[0].long()
        ramp, sizes = torch.linspace(0.02, 3.0, order.numel(), device=DEV), torch.exp2(torch.linspace(-30, 10, order.numel(), device=DEV))
        c.ks[0, order] = (ramp if up > 0 else ramp.flip(0))[:, None] * 0.004
        c.vs[0, order] = (sizes if up > 0 else sizes.flip(0))[:, None]
        i = np.arange(2000) // 16
        o = c.table[0].long().cpu().numpy()
        c.old[0] = [(c.old[0][0][0], f64(c.ks)[0, o][i]), (c.old[0][1][0], f64(c.vs)[0, o][i])]
        c.run()
        c.check(norm=False)


def test_scales_of_zero():
    c = Case(9, [300], [2], 8, 1, 128)
    order = c.table[0].long().cpu().numpy()
    c.ks[0, int(order[1])] = 0.0
    c.vs[0, int(order[2])] = 0.0
    i = np.arange(300) // 64
    c.old[0] = [(c.old[0][0][0], f64(c.ks)[0, order][i]), (c.old[0][1][0], f64(c.vs)[0, order][i])]
    c.run()
    c.check()
    c.vs.zero_()
    c.run()
    torch.cuda.synchronize()
    assert (f64(c.o) == 0).all()


def test_slots_layers_and_a_sequence_read_twice():
    c = Case(10, [300, 120, 300], [2, 5, 1], layers=3, layer=1, slots=[4, 0, 4])
    c.run()
    c.check()


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (256, "fp16")])
def test_values_behind_a_row_cannot_change_it(D, dtype):
    c = Case(11, [200], [140], 4, 2, D, 32, dtype)
    a = c.run().clone()
    c.check()
    pages = c.table[0].long()
    for p in (199, 150):   # codes NaN in K and V at position p: rows that see it change, the others do not
        for pool in (c.k, c.v):
            pool.view(torch.uint8)[0, pages[p // 32], p % 32, 1, 3:7] = 0x7F if p == 150 else 0xFF
        b = c.run().clone()
        torch.cuda.synchronize()
        row = p - 60
        assert torch.equal(a[:row], b[:row])
        assert torch.equal(a[:, :2], b[:, :2])                       # the other KV head's
        assert b[row:, 2:].isnan().all()                             # NaN among the scores


@pytest.mark.parametrize("L,n", [(200, 140), (3000, 5), (128, 128), (20000, 1), (20000, 40)])
@pytest.mark.parametrize("D", [64, 256])
def test_values_that_are_nan_show_in_their_columns(L, n, D):
    c = Case(12, [L], [n], 4, 2, D, 64)
    a = c.run().clone()
    c.check()
    pages = c.table[0].long()
    for p, d in ((L - 1, 5), (max(0, L - n + n // 2), 33), (L // 3, 60)):
        c.v.view(torch.uint8)[0, pages[p // 64], p % 64, 1, d] = 0x7F
    b = c.run()
    torch.cuda.synchronize()
    want = torch.zeros_like(b, dtype=torch.bool)
    for p, d in ((L - 1, 5), (max(0, L - n + n // 2), 33), (L // 3, 60)):
        want[max(0, p - (L - n)):, 2:, d] = True
    assert torch.equal(b.isnan(), want)
    assert torch.equal(a[~want], b[~want])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("L", [64, 3000, 40000])
def test_a_query_that_is_not_a_number_gives_none(bad, L):
    c = Case(13, [L], [3])
    a = c.run().clone()
    c.q[1, 4, 17] = bad
    b = c.run()
    torch.cuda.synchronize()
    assert b[1, 4].isnan().all()
    b[1, 4] = a[1, 4]
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunks_over_many_tiles(D, dtype):
    c = Case(22, [2500, 900], [70, 33], 16, 2, D, 64, dtype)
    c.run()
    c.check()


@pytest.mark.parametrize("rows", [8, 9, 16, 17, 40])
def test_row_counts_at_which_the_kernel_changes(rows):
    c = Case(23, [1000, 300, 40], [rows, rows - 1, 1], 1, 1, 128, 32, "fp16")
    c.run()
    c.check()


# units that are not cut, and next to those that are: as many as there are CTAs and one more, the longest at
# eight tiles above an equal share and beyond, sequences without rows among them, several row tiles
@pytest.mark.parametrize("lens,counts,Hq,Hkv", [
    ([700] * 40, [1] * 40, 8, 2), ([300] * 76, [1] * 76, 4, 2), ([300] * 77, [1] * 77, 4, 2),
    ([640], [1], 4, 1), ([641], [1], 4, 1), ([769], [1], 4, 1), ([3000, 2500, 0, 2900] * 30, [1, 2, 0, 1] * 30, 2, 1),
    ([3000] + [100] * 149, [1] * 150, 2, 1), ([400, 90, 350], [40, 33, 0], 8, 1), ([700, 660], [150, 130], 16, 2),
    ([0] * 5, [0] * 5, 2, 1), ([0, 5, 0], [3, 0, 0], 2, 1)])
def test_units_that_are_runs(lens, counts, Hq, Hkv):
    c = Case(24, lens, counts, Hq, Hkv, 128, 32)
    c.run()
    c.check()


def test_a_long_cache():
    c = Case(14, [131000], [3], 4, 1, 256, 128)
    c.run()
    c.check()


def test_many_sequences_attend():
    rng = np.random.default_rng(15)
    c = Case(15, rng.integers(0, 60, 1024).tolist(), rng.integers(0, 3, 1024).tolist(), 2, 1, 64, 16)
    c.run()
    c.check()


def test_offsets_beyond_31_bits():
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 20 GB")
    c = Case(16, [500, 77], [2, 2], 4, 2, 256, 256)
    P = (1 << 31) // 256 // 4                                        # 2 G rows in 4 layers, of 512 bytes: 1 TB would be all;
    P = min(P, 9000)                                                 # 9,000 pages of 256 rows in 2 layers are 2.4 GB
    layers = 2
    big = [torch.empty(layers, P, 256, 2, 256, dtype=torch.uint8, device=DEV).view(F8) for _ in "kv"]
    scales = [torch.full((layers, P, 2), float("nan"), device=DEV) for _ in "kv"]
    move = {int(p): P - 1 - i for i, p in enumerate(c.table[c.table >= 0].tolist())}
    for pool, small, sc, ssc in ((big[0], c.k, scales[0], c.ks), (big[1], c.v, scales[1], c.vs)):
        for a, b in move.items():
            pool.view(torch.uint8)[1, b] = small.view(torch.uint8)[0, a]
            sc[1, b] = ssc[0, a]
    table = i32([[move.get(p, -1) for p in row] for row in c.table.tolist()])
    cache = moe.make_attn_qcache(*big, *scales, i32([1] * P), table, c.slot_lens, c.status)
    ws = torch.zeros(moe.attn_qcache_attend_workspace_bytes(cache, 2, 4, 2, 4), dtype=torch.uint8, device=DEV)
    moe.attn_qcache_attend(cache, 1, c.q, i32(c.off.tolist()), 2, 2, ws, c.o)
    c.check()


def test_calls_repeat_exactly_and_replay_from_a_graph():
    c = Case(17, [4000, 900, 10], [5, 3, 10])
    first = c.run().clone()
    for _ in range(5):
        assert torch.equal(c.run(), first)
    off = i32(c.off.tolist())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                moe.attn_qcache_attend(c.cache, 0, c.q, off, 3, c.max_rows, c.ws, c.o)
    torch.cuda.synchronize()
    for gain in (1.0, 2.0):
        c.q.mul_(gain)
        c.o.zero_()
        g.replay()
        c.check()
    c.slot_lens[1] = c.lens[1] = 300          # the lengths are the device's: the same graph follows them
    c.old[1] = [(a[:300], b[:300]) for a, b in c.old[1]]
    g.replay()
    c.check()


def test_two_streams_with_a_workspace_each():
    c, d = Case(18, [3000, 100], [4, 2]), Case(19, [50, 7000], [2, 4], dtype="fp16")
    a, b = c.run().clone(), d.run().clone()
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        c.run(stream=s)
        d.run(stream=t)
    torch.cuda.synchronize()
    assert torch.equal(c.o, a) and torch.equal(d.o, b)
    c.check()


@pytest.mark.parametrize("what", ["slot", "slot_low", "offset", "order", "max_rows", "length", "page"])
def test_device_checks(what):
    c = Case(20, [300, 200, 100], [3, 3, 3])
    a = c.run().clone()
    off, slots, mr = c.off.tolist(), [0, 1, 2], 3
    if what == "slot":
        slots[1] = 3
    elif what == "slot_low":
        slots[1] = -1
    elif what == "offset":
        off[3] = 10
    elif what == "order":
        off = [0, 3, 2, 9]
    elif what == "max_rows":
        mr = 2
    elif what == "length":
        c.slot_lens[1] = 1 << 20
    else:
        c.table[1, 1] = c.k.shape[1]
    moe.attn_qcache_attend(c.cache, 0, c.q, i32(off), 3, mr, c.ws, c.o, slots=i32(slots))
    torch.cuda.synchronize()
    assert int(c.status[0]) == moe.MOE_ERR_DEVICE_BOUNDS
    if what in ("slot", "slot_low", "length", "page"):               # the others are as they were
        assert torch.equal(c.o[:3], a[:3]) and torch.equal(c.o[6:], a[6:])


def test_binding_refusals():
    c = Case(21, [300], [3])
    off = i32([0, 3])
    for bad in (dict(q=c.q.float()), dict(q=c.q[:, :, :128]), dict(q=c.q.cpu()), dict(off=off.long()), dict(ws=c.ws.cpu()),
                dict(o=c.o.half()), dict(o=c.o[:2])):
        a = {**dict(q=c.q, off=off, ws=c.ws, o=c.o), **bad}
        with pytest.raises(ValueError):
            moe.attn_qcache_attend(c.cache, 0, a["q"], a["off"], 1, 3, a["ws"], a["o"])
    with pytest.raises(moe.MoeError):
        moe.attn_qcache_attend(c.cache, 0, c.q, off, 1, 3, c.ws, c.q)
    with pytest.raises(ValueError):
        moe.make_attn_qcache(c.k, c.v, c.ks[:, :-1], c.vs, c.refs, c.table, c.slot_lens, c.status)
    with pytest.raises(ValueError):
        moe.make_attn_qcache(c.k.view(torch.uint8), c.v, c.ks, c.vs, c.refs, c.table, c.slot_lens, c.status)
    with pytest.raises(ValueError):
        moe.make_attn_cache(c.k, c.v, c.refs, c.table, c.slot_lens, c.status)


# ---------------------------------------------------------- the operators together

def test_steps_of_a_model():
    # prompts in chunks, then tokens one by one: q and K turned, appended and attended; a fork; a cut
    t = Twin(32, 2, 128, "bf16", pages=60, slots=4, max_pages=16, layers=2)
    rot, w = moe.make_rotary(64, base=1e6), rates(64, base=1e6)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    Hq = 8
    for step, counts in enumerate([[70, 33], [1, 5], [1, 1], [40, 1]]):
        N = sum(counts)
        kn, vn, q = t.normal(2, N, 2, 128), t.normal(2, N, 2, 128), t.normal(2, N, Hq, 128)
        off = i32([0, counts[0], N])
        L = t.lens[:2].tolist()
        pos = [L[0] + i for i in range(counts[0])] + [L[1] + i for i in range(counts[1])]
        moe.attn_qcache_append(t.cache, rot, kn, vn, off, 2, ws)
        o, turned = torch.empty_like(q), torch.empty_like(q)
        for l in range(2):
            moe.attn_rotary(rot, q[l], i32(pos), turned[l])
            moe.attn_qcache_attend(t.cache, l, turned[l], off, 2, max(counts), ws, o[l])
        torch.cuda.synchronize()
        assert int(t.status[0]) == 0
        m = QPages(*[f64(x) for x in (t.k, t.v, t.ks, t.vs)], *[x.cpu().numpy() for x in (t.refs, t.table, t.lens)])
        for l in range(2):
            for s, lo, n in ((0, 0, counts[0]), (1, counts[0], counts[1])):
                ref, mass, _ = attend(f64(turned[l, lo:lo + n]), *m.values(s, l))
                assert (np.abs(f64(o[l, lo:lo + n]) - ref) <= mass * 2.0 ** -6 + 2.0 ** -8).all()
        if step == 1:
            moe.attn_qcache_fork(t.cache, i32([0]), i32([3]), 1, ws)
            moe.attn_qcache_trim(t.cache, None, i32([60, 20]), 2)
    assert t.lens.tolist() == [101, 22, 0, 71]
