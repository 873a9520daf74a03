"""GPU parity of rotary positions (attn_rotary, attn_cache_append_rotary)
against the fp64 oracle.

Tolerance, from the arithmetic: with u half a step of the type (bf16 2^-8, fp16
2^-11, and half of fp16's least step 2^-24), o is rounded once: u |o|.  The angle: the rate is off
by 2^-53 of itself (a few: pow and two products) or 2^-64 turns, times the
position; what it is beyond a quarter turn is rounded to 2^-24 of itself, an eighth of
a turn at most, and multiplied by 2 pi: below 2^-22.3 radians.  cos and sin are off by 2^-23, the two products and
their sum by 2^-24 each, the factor by 2^-24: all in all (|x| + |y|) |factor|
(2^-20 + |p| 2^-49).
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle.rotary import rates, rotate
from oracle.tree import Pages

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import bit_grouped_expert_gb300 as moe  # noqa: E402

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
LONG = dict(base=500000.0, stretch=16.0, low_turns=1.0, high_turns=32.0, original_len=4096)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_grouped_expert_gb300 import build
    build.build()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def normal(seed, *shape, dtype="bf16"):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.empty(shape, dtype=TYPES[dtype], device=DEV).normal_(generator=g)


def f64(t):
    return t.double().cpu().numpy()


def plan(dim, inter=False, factor=1.0, **kw):
    return moe.make_rotary(dim, interleaved=inter, factor=factor, **kw), rates(dim, **{**dict(base=10000.0), **kw})


def bound(x, ref, w, positions, dtype, inter, factor):
    h = len(w)
    size = np.zeros_like(ref)
    pairs = np.abs(x)
    a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if inter else (slice(0, h), slice(h, 2 * h))
    size[..., a] = size[..., b] = pairs[..., a] + pairs[..., b]
    p = np.abs(np.asarray(positions, np.float64))[:, None, None]
    return HALF[dtype] * np.abs(ref) + 2.0 ** -25 * (dtype == "fp16") + size * abs(factor) * (2.0 ** -20 + p * 2.0 ** -49)


def check(o, x, w, positions, dtype, inter=False, factor=1.0):
    ref = rotate(f64(x), positions, w, inter, factor)
    err = np.abs(f64(o) - ref)
    lim = bound(f64(x), ref, w, positions, dtype, inter, factor)
    assert (err <= lim * (1 + 1e-6)).all(), float((err - lim).max())
    np.testing.assert_array_equal(f64(o)[..., 2 * len(w):], f64(x)[..., 2 * len(w):])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,dim", [(64, 16), (64, 48), (64, 64), (128, 32), (128, 128), (256, 64), (256, 208), (256, 256)])
def test_layouts_and_parts_of_a_head(D, dim, inter, dtype):
    rot, w = plan(dim, inter)
    x = normal(1, 7, 5, D, dtype=dtype)
    positions = [0, 1, 2, 77, 5000, 131071, 1000003]
    o = torch.empty_like(x)
    moe.attn_rotary(rot, x, i32(positions), o)
    check(o, x, w, positions, dtype, inter)


@pytest.mark.parametrize("n,heads", [(1, 1), (1, 16), (1, 3), (2, 64), (33, 2), (257, 9), (3000, 1)])
def test_sizes(n, heads):
    rot, w = plan(64)
    x = normal(n, n, heads, 128)
    positions = np.random.default_rng(n).integers(0, 100000, n).tolist()
    o = torch.empty_like(x)
    moe.attn_rotary(rot, x, i32(positions), o)
    check(o, x, w, positions, "bf16")


@pytest.mark.parametrize("kw", [LONG, dict(stretch=8.0), dict(base=1e6, stretch=4.0, low_turns=0.0, high_turns=2.5,
                                                              original_len=1000)])
def test_stretched_rates(kw):
    rot, w = plan(128, factor=1.2, **kw)
    x = normal(5, 9, 4, 128, dtype="fp16")
    positions = [0, 5, 100, 4095, 4096, 60000, 65535, 1 << 20, (1 << 20) + 1]
    o = torch.empty_like(x)
    moe.attn_rotary(rot, x, i32(positions), o)
    check(o, x, w, positions, "fp16", factor=1.2)


def test_the_farthest_positions():
    rot, w = plan(64, True)
    x = normal(6, 4, 2, 64, dtype="fp16")
    positions = [2 ** 31 - 1, -2 ** 31, -1, 2 ** 30 + 12345]
    o = torch.empty_like(x)
    moe.attn_rotary(rot, x, i32(positions), o)
    check(o, x, w, positions, "fp16", True)


def test_turning_back_is_the_gradient():
    # L = <y, R_p x>: dL/dx = R_-p y, against differences of the formula
    w = rates(16)
    rng = np.random.default_rng(3)
    x, y, p = rng.normal(size=(1, 1, 64)), rng.normal(size=(1, 1, 64)), [12345]
    back = rotate(y, [-p[0]], w)
    for d in range(64):
        e = np.zeros_like(x)
        e[..., d] = 1e-3
        slope = ((rotate(x + e, p, w) - rotate(x - e, p, w)) * y).sum() / 2e-3
        assert abs(slope - back[0, 0, d]) < 1e-9
    rot, _ = plan(16)
    t = torch.from_numpy(y).to(DEV).to(torch.float16)
    o = torch.empty_like(t)
    moe.attn_rotary(rot, t, i32([-p[0]]), o)
    check(o, t, w, [-p[0]], "fp16")


def test_rows_apart_in_place_and_nothing_else_written():
    rot, w = plan(64)
    wide = normal(8, 11, 4 * 128 + 24)
    was = wide.clone()
    positions = list(range(100, 111))
    x = wide[:, 8:8 + 512].unflatten(1, (4, 128))
    assert x.data_ptr() % 16 == 0
    o = torch.empty(11, 4, 128, dtype=torch.bfloat16, device=DEV)
    moe.attn_rotary(rot, x, i32(positions), o)
    check(o, x, w, positions, "bf16")
    assert torch.equal(wide, was)
    moe.attn_rotary(rot, x, i32(positions), x)
    assert torch.equal(x, o)
    assert torch.equal(wide[:, :8], was[:, :8]) and torch.equal(wide[:, 520:], was[:, 520:])
    out = torch.full((11, 600), float("nan"), dtype=torch.bfloat16, device=DEV)
    moe.attn_rotary(rot, was[:, 8:520].unflatten(1, (4, 128)), i32(positions), out[:, :512].unflatten(1, (4, 128)))
    assert torch.equal(out[:, :512].unflatten(1, (4, 128)), o) and out[:, 512:].isnan().all()


def test_offsets_beyond_31_bits():
    rows, row = 5000, 64 * 256 * 32  # 5.2 GB apart
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 6 GB")
    wide = torch.zeros(rows, row, dtype=torch.bfloat16, device=DEV)
    x = wide[:, :512].unflatten(1, (2, 256))
    x.copy_(normal(9, rows, 2, 256))
    rot, w = plan(256)
    positions = (np.arange(rows) * 7).tolist()
    o = torch.empty(rows, 2, 256, dtype=torch.bfloat16, device=DEV)
    moe.attn_rotary(rot, x, i32(positions), o)
    check(o[-5:], x[-5:], w, positions[-5:], "bf16")
    check(o[:5], x[:5], w, positions[:5], "bf16")


def test_values_that_are_not_finite_stay_in_their_pairs():
    rot, w = plan(32, True)
    x = normal(10, 3, 2, 64)
    x[1, 0, 4], x[1, 0, 50], x[2, 1, 7] = float("nan"), float("inf"), float("inf")
    o = torch.empty_like(x)
    moe.attn_rotary(rot, x, i32([3, 4, 5]), o)
    bad = ~torch.isfinite(o)
    want = torch.zeros_like(bad)
    want[1, 0, 4:6] = want[1, 0, 50] = want[2, 1, 6:8] = True
    assert torch.equal(bad, want)


def test_another_stream_and_a_graph():
    rot, w = plan(64)
    x, positions, o = normal(11, 40, 16, 256), i32([0] * 40), torch.zeros(40, 16, 256, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            moe.attn_rotary(rot, x, positions, o)
            moe.attn_rotary(rot, o, positions, o)  # a call that depends on the one before
    torch.cuda.synchronize()
    for k in (3, 90):
        positions.fill_(k)
        g.replay()
        torch.cuda.synchronize()
        once = torch.empty_like(x)
        moe.attn_rotary(rot, x, positions, once)
        check(once, x, w, [k] * 40, "bf16")
        check(o, once, w, [k] * 40, "bf16")


def test_binding_refusals():
    rot, _ = plan(64)
    x, p = normal(1, 4, 2, 128), i32([0, 1, 2, 3])
    o = torch.empty_like(x)
    for a in (dict(x=x.float()), dict(x=x[:, :, ::2]), dict(x=x.transpose(0, 1)), dict(p=p.long()), dict(p=p[:3]),
              dict(o=o[:3]), dict(o=o.half()), dict(x=x.cpu()), dict(p=p.cpu()), dict(x=x.reshape(4, 256))):
        b = {**dict(x=x, p=p, o=o), **a}
        with pytest.raises((ValueError, RuntimeError)):
            moe.attn_rotary(rot, b["x"], b["p"], b["o"])
    flat = normal(2, 4 * 256 + 8)
    with pytest.raises(moe.MoeError):  # onto itself, a little further on
        moe.attn_rotary(rot, flat[:1024].reshape(4, 2, 128), p, flat[8:].reshape(4, 2, 128))
    with pytest.raises(moe.MoeError):  # rows that lie over one another
        moe.attn_rotary(rot, x[:1].expand(4, 2, 128), p, o)
    moe.attn_rotary(rot, x[:0], p[:0], o[:0])


# ------------------------------------------------------- appending to the 16-bit cache

class Twin:
    """A cache on the GPU and the oracle's copy of it."""

    def __init__(self, page=16, heads=2, dim=64, dtype="bf16", pages=40, slots=6, max_pages=12, layers=2):
        self.shape, self.dtype = (layers, heads, dim), dtype
        self.k, self.v = (normal(i, layers, pages, page, heads, dim, dtype=dtype) for i in (1, 2))
        self.refs, self.lens = i32([0] * pages), i32([0] * slots)
        self.table, self.status = torch.full((slots, max_pages), -1, dtype=torch.int32, device=DEV), i32([0] * 4)
        self.cache = moe.make_attn_cache(self.k, self.v, self.refs, self.table, self.lens, self.status)
        self.model = Pages(f64(self.k), f64(self.v), *[t.cpu().numpy().copy() for t in (self.refs, self.table, self.lens)])
        self.turned = np.zeros(self.model.k.shape[:3], bool)
        self.calls = 0

    def append(self, rot, w, counts, slots=None, keep=None, path=None, inter=False, factor=1.0):
        layers, heads, dim = self.shape
        off = np.concatenate([[0], np.cumsum(counts)])
        N, B = int(off[-1]), len(counts)
        self.calls += 1
        kn, vn = (normal(100 * self.calls + i, layers, N, heads, dim, dtype=self.dtype) for i in (1, 2))
        ws = torch.full((moe.attn_cache_append_workspace_bytes(self.cache, B, N),), 0xFF, dtype=torch.uint8, device=DEV)
        opt = {n: None if v is None else i32(v) for n, v in (("slots", slots), ("n_keep", keep), ("path", path))}
        moe.attn_cache_append_rotary(self.cache, rot, kn, vn, i32(off.tolist()), B, ws, **opt)
        jobs, lim = [], []
        for b in range(B):
            s, n = b if slots is None else slots[b], counts[b] if keep is None else keep[b]
            pick = [off[b] + (i if path is None else path[b][i]) for i in range(n)]
            L = int(self.model.lens[s])
            pos = list(range(L, L + n))
            x = f64(kn[:, pick])
            kr = np.stack([rotate(x[l], pos, w, inter, factor) for l in range(layers)]) if n else x
            lim.append((s, L, np.stack([bound(x[l], kr[l], w, pos, self.dtype, inter, factor) for l in range(layers)])
                        if n else x))
            jobs.append((s, kr, f64(vn[:, pick])))
        self.model.append(jobs)
        torch.cuda.synchronize()
        assert int(self.status[0]) == 0
        for name in ("refs", "table", "lens"):
            np.testing.assert_array_equal(getattr(self, name).cpu().numpy(), getattr(self.model, name), err_msg=name)
        np.testing.assert_array_equal(f64(self.v), self.model.v)
        got = f64(self.k)
        allow = np.zeros(got.shape)
        for s, L, e in lim:
            for i in range(e.shape[1]):
                page, at = self.model.table[s, (L + i) // self.model.page], (L + i) % self.model.page
                allow[:, page, at] = e[:, i]
        assert (np.abs(got - self.model.k) <= allow * (1 + 1e-6)).all()  # all other rows: exactly as they were
        self.model.k = got


@pytest.mark.parametrize("page,heads,dim,dtype,rdim,inter", [
    (16, 2, 64, "bf16", 64, False), (64, 1, 128, "fp16", 32, True), (32, 3, 256, "bf16", 256, True),
    (128, 8, 64, "fp16", 16, False), (256, 2, 256, "bf16", 64, False)])
def test_appends_turn_k_by_the_place_it_goes_to(page, heads, dim, dtype, rdim, inter):
    rot, w = plan(rdim, inter, 1.1, **LONG)
    kw = dict(inter=inter, factor=1.1)
    t = Twin(page, heads, dim, dtype)
    t.append(rot, w, [page, 1, 0, 2 * page + 3], **kw)
    t.append(rot, w, [5, page - 1], slots=[3, 1], keep=[2, page - 1],
             path=[[4, 0] + [0] * page, list(range(page - 1)) + [0] * 3], **kw)
    ws = torch.zeros(moe.attn_cache_fork_workspace_bytes(t.cache, 2), dtype=torch.uint8, device=DEV)
    moe.attn_cache_fork(t.cache, i32([3, 3]), i32([4, 5]), 2, ws)
    t.model.fork([(3, 4), (3, 5)])
    t.append(rot, w, [1, 2, 1], slots=[5, 4, 3], **kw)  # rows of copied pages are not turned again


def test_a_chunk_of_many_rows():
    rot, w = plan(64)
    t = Twin(64, 2, 256, "bf16", pages=60, layers=5, max_pages=20)
    t.append(rot, w, [700, 3, 400])
    t.append(rot, w, [1, 500, 100])


def test_append_agrees_with_turning_first():
    # the same rows turned by attn_rotary and appended as they are: bit for bit
    rot, _ = plan(128, True)
    a, b = Twin(32, 4, 128, "fp16", layers=1), Twin(32, 4, 128, "fp16", layers=1)
    kn, vn = normal(20, 1, 50, 4, 128, dtype="fp16"), normal(21, 1, 50, 4, 128, dtype="fp16")
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)
    moe.attn_cache_append_rotary(a.cache, rot, kn, vn, i32([0, 30, 50]), 2, ws)
    turned = torch.empty_like(kn[0])
    moe.attn_rotary(rot, kn[0], i32(list(range(30)) + list(range(20))), turned)
    moe.attn_cache_append(b.cache, turned[None], vn, i32([0, 30, 50]), 2, ws)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and torch.equal(a.table, b.table)


def test_an_append_that_fails_changes_nothing():
    rot, w = plan(64)
    t = Twin(max_pages=3)
    t.append(rot, w, [20, 17])
    was = [x.clone() for x in (t.k, t.v, t.refs, t.table, t.lens)]
    kn, vn = normal(30, 2, 34, 2, 64), normal(31, 2, 34, 2, 64)
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)
    moe.attn_cache_append_rotary(t.cache, rot, kn, vn, i32([0, 2, 34]), 2, ws)  # no room in the second's table
    torch.cuda.synchronize()
    assert int(t.status[0]) == moe.MOE_ERR_DEVICE_BOUNDS
    assert all(torch.equal(x, y) for x, y in zip(was, (t.k, t.v, t.refs, t.table, t.lens)))
    with pytest.raises(moe.MoeError):  # more is turned than a head has
        moe.attn_cache_append_rotary(t.cache, plan(128)[0], kn, vn, i32([0, 2, 34]), 2, ws)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("stretch", [1.0, 32.0, 1e4, 1e7])
def test_small_angles_keep_their_bits(stretch, inter, dtype):
    # Pairs (x, 0) become (x cos a, x sin a), so that the second value is as exact as a itself: the fraction of a turn is
    # rounded to 2^-24 of itself, then multiplied by 2 pi (2^-24, the constant 2^-25); the series, the factor
    # and the product with x another 2^-24 each, the rate 2^-50 and 2^-64 turns of 1 / (turns a position): 2^-21 together.
    D = 256
    rot, w = plan(D, inter, base=1e6, stretch=stretch)
    x = normal(12, 8, 2, D, dtype=dtype).abs() + 0.5
    second = slice(1, D, 2) if inter else slice(D // 2, D)
    x[..., second] = 0.0
    positions = [0, 1, -1, 10, -37, 1000, 4097, -100000]
    o = torch.empty_like(x)
    moe.attn_rotary(rot, x, i32(positions), o)
    ref = rotate(f64(x), positions, w, inter)[..., second]
    small = np.abs(np.outer(positions, w))[:, None, :] < np.pi / 4   # beyond, the quarter turns' own errors count
    lim = np.abs(ref) * (HALF[dtype] + 2.0 ** -21 + 2.0 ** -64 * 2 * np.pi / w) + 2.0 ** -25 * (dtype == "fp16")
    err = np.abs(f64(o)[..., second] - ref)
    assert (err <= lim)[np.broadcast_to(small, err.shape)].all(), float((err / np.maximum(lim, 1e-300) * small).max())
    check(o, x, w, positions, dtype, inter)
