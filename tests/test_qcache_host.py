"""Host checks of the rotary and 8-bit cache entry points (every call here is
refused on the host, or has nothing to do, before anything is enqueued), and
their oracles against closed forms."""
from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest

import bit_grouped_expert_gb300 as moe
from oracle.qcache import QPages, attend, nearest, scale_of
from oracle.rotary import rates, rotate

A = 0x10000000  # fake, aligned device addresses


@pytest.fixture(scope="module")
def lib():
    from bit_grouped_expert_gb300 import build
    build.build()
    return moe.lib()


def _cache(**kw):
    d = dict(k_d=A, v_d=2 * A, k_scale_d=14 * A, v_scale_d=15 * A, refs_d=3 * A, table_d=4 * A, lens_d=5 * A,
             status_d=6 * A, n_layers=2, n_pages=100, page_size=64, n_kv_heads=2, head_dim=256, n_slots=8, max_pages=20)
    d.update(kw)
    return moe.attn_qcache(**d)


def _table(lib, dim=64, inter=0, **kw):
    cfg = moe.attn_rotary_config(dim, inter, *(kw.get(n, d) for n, d in
                                               (("base", 10000.0), ("stretch", 1.0), ("low", 0.0), ("high", 0.0),
                                                ("original", 0.0), ("factor", 1.0))))
    t = moe.attn_rotary_table()
    return lib.attn_rotary_plan(ctypes.byref(cfg), ctypes.byref(t)), t


BAD_CACHES = [(dict(k_d=None), moe.MOE_ERR_INVALID_ARGUMENT), (dict(k_scale_d=None), moe.MOE_ERR_INVALID_ARGUMENT),
              (dict(v_scale_d=None), moe.MOE_ERR_INVALID_ARGUMENT), (dict(lens_d=None), moe.MOE_ERR_INVALID_ARGUMENT),
              (dict(n_pages=0), moe.MOE_ERR_INVALID_ARGUMENT), (dict(page_size=48), moe.MOE_ERR_UNSUPPORTED),
              (dict(page_size=512), moe.MOE_ERR_UNSUPPORTED), (dict(head_dim=96), moe.MOE_ERR_UNSUPPORTED),
              (dict(n_kv_heads=257), moe.MOE_ERR_UNSUPPORTED), (dict(n_pages=1 << 25), moe.MOE_ERR_UNSUPPORTED),
              (dict(v_d=A + 8), moe.MOE_ERR_MISALIGNED), (dict(v_scale_d=A + 4), moe.MOE_ERR_MISALIGNED)]


@pytest.mark.parametrize("change,want", BAD_CACHES)
def test_bad_caches_are_refused_by_every_entry_point(lib, change, want):
    c = ctypes.byref(_cache(**change))
    assert lib.attn_qcache_append(c, None, 7 * A, 8 * A, moe.MOE_BF16, None, 9 * A, None, None, 0, 3, 30, 12 * A, 1 << 20,
                                  0) == want
    assert lib.attn_qcache_fork(c, A, A, 2, A, 1 << 20, 0) == want
    assert lib.attn_qcache_trim(c, A, A, 2, 0) == want
    assert lib.attn_qcache_attend(c, 0, A, moe.MOE_BF16, None, A, 1, 4, 4, 16, ctypes.c_float(0), A, 1 << 30, A, 0) == want
    assert lib.attn_qcache_append_workspace_bytes(c, 1, 1) == 0
    assert lib.attn_qcache_fork_workspace_bytes(c, 1) == 0
    assert lib.attn_qcache_attend_workspace_bytes(c, 1, 1, 1, 16) == 0


def test_append_host_checks(lib):
    ok, table = _table(lib)
    assert ok == moe.MOE_OK

    def call(c=None, table=table, dtype=moe.MOE_BF16, B=3, rows=30, ws=None, stride=4, **kw):
        c = ctypes.byref(_cache() if c is None else c)
        a = {**dict(k=7 * A, v=8 * A, slots=None, off=9 * A, keep=10 * A, path=11 * A, ws=12 * A), **kw}
        need = lib.attn_qcache_append_workspace_bytes(c, B, rows) if ws is None else ws
        return lib.attn_qcache_append(c, None if table is None else ctypes.byref(table), a["k"], a["v"], dtype, a["slots"],
                                      a["off"], a["keep"], a["path"], stride, B, rows, a["ws"], need, 0)

    assert lib.attn_qcache_append(None, None, A, A, 0, None, A, None, None, 0, 1, 1, A, 1 << 20, 0) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(B=0) == moe.MOE_OK
    assert call(B=0, table=None) == moe.MOE_OK
    assert call(B=-1) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(rows=-1) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(k=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(off=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(keep=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(stride=0) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(dtype=2) == moe.MOE_ERR_UNSUPPORTED
    assert call(B=1025, ws=1 << 30) == moe.MOE_ERR_UNSUPPORTED
    assert call(v=A + 2) == moe.MOE_ERR_MISALIGNED
    pool = 2 * 100 * 64 * 512  # bytes of K's codes
    assert call(k=A + pool - 16) == moe.MOE_ERR_INVALID_ARGUMENT  # rows inside the pool
    assert call(v=2 * A) == moe.MOE_ERR_INVALID_ARGUMENT
    need = lib.attn_qcache_append_workspace_bytes(ctypes.byref(_cache()), 3, 30)
    assert need > 0 and call(ws=need - 1) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    assert call(c=_cache(head_dim=64), table=_table(lib, 128)[1]) == moe.MOE_ERR_UNSUPPORTED  # more than a head has
    bad = moe.attn_rotary_table()
    assert call(table=bad) == moe.MOE_ERR_UNSUPPORTED  # never planned


def test_fork_and_trim_host_checks(lib):
    c = ctypes.byref(_cache())
    need = lib.attn_qcache_fork_workspace_bytes(c, 4)

    def fork(src=A, dst=2 * A, n=4, ws=3 * A, nb=need):
        return lib.attn_qcache_fork(c, src, dst, n, ws, nb, 0)

    assert fork(n=0, src=None) == moe.MOE_OK
    assert fork(n=-1) == moe.MOE_ERR_INVALID_ARGUMENT
    assert fork(dst=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert fork(n=1025, nb=1 << 20) == moe.MOE_ERR_UNSUPPORTED
    assert fork(src=A + 4) == moe.MOE_ERR_MISALIGNED
    assert fork(nb=need - 1) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    assert lib.attn_qcache_trim(c, None, None, 0, 0) == moe.MOE_OK
    assert lib.attn_qcache_trim(c, None, None, 1, 0) == moe.MOE_ERR_INVALID_ARGUMENT
    assert lib.attn_qcache_trim(c, None, A, 1025, 0) == moe.MOE_ERR_UNSUPPORTED
    assert lib.attn_qcache_trim(c, A + 4, A, 1, 0) == moe.MOE_ERR_MISALIGNED


def test_attend_host_checks(lib):
    def call(c=None, layer=0, dtype=moe.MOE_FP16, B=2, n=10, mx=8, Hq=16, scale=0.0, nb=None, **kw):
        c = ctypes.byref(_cache() if c is None else c)
        a = {**dict(q=7 * A, slots=None, off=10 * A, ws=12 * A, o=13 * A), **kw}
        need = lib.attn_qcache_attend_workspace_bytes(c, B, n, mx, Hq) if nb is None else nb
        return lib.attn_qcache_attend(c, layer, a["q"], dtype, a["slots"], a["off"], B, n, mx, Hq, ctypes.c_float(scale),
                                      a["ws"], need, a["o"], 0)

    assert call(B=0) == moe.MOE_OK
    assert call(n=0, q=None) == moe.MOE_OK
    assert call(layer=2) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(layer=-1) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(B=-1) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(mx=0) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(Hq=0) == moe.MOE_ERR_INVALID_ARGUMENT
    for scale in (-0.5, float("nan"), float("inf")):
        assert call(scale=scale) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(off=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(o=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(dtype=2) == moe.MOE_ERR_UNSUPPORTED
    assert call(Hq=15, nb=1 << 30) == moe.MOE_ERR_UNSUPPORTED
    assert call(Hq=258, nb=1 << 30) == moe.MOE_ERR_UNSUPPORTED  # 129 query heads per KV head
    assert call(B=1025, nb=1 << 30) == moe.MOE_ERR_UNSUPPORTED
    assert call(n=1 << 27, nb=1 << 60) == moe.MOE_ERR_UNSUPPORTED
    assert call(q=7 * A + 2) == moe.MOE_ERR_MISALIGNED
    assert call(slots=A + 4) == moe.MOE_ERR_MISALIGNED
    for x in (7 * A + 16, A + 4096, 2 * A, 14 * A, 15 * A + 64):  # the output over the queries, the pool or the scales
        assert call(o=x) == moe.MOE_ERR_INVALID_ARGUMENT
    for mx in (1, 8):  # few rows and whole matrices
        need = lib.attn_qcache_attend_workspace_bytes(ctypes.byref(_cache()), 2, 10, mx, 16)
        assert need > 0 and call(mx=mx, nb=need - 1) == moe.MOE_ERR_WORKSPACE_TOO_SMALL


def test_rotary_host_checks(lib):
    assert lib.attn_rotary_plan(None, None) == moe.MOE_ERR_INVALID_ARGUMENT
    for kw in (dict(base=0.0), dict(base=-2.0), dict(base=float("inf")), dict(stretch=0.0), dict(stretch=float("nan")),
               dict(factor=float("inf")), dict(low=2.0, high=1.0, original=10.0), dict(low=-1.0, high=1.0, original=10.0),
               dict(high=1.0, original=0.0), dict(low=1.0, high=0.0), dict(inter=2)):
        assert _table(lib, **kw)[0] == moe.MOE_ERR_INVALID_ARGUMENT, kw
    for dim in (0, 8, 24, 272, -16):
        assert _table(lib, dim)[0] == moe.MOE_ERR_UNSUPPORTED
    table = _table(lib, 128)[1]

    def call(table=table, x=A, xs=512, dtype=0, p=2 * A, n=4, H=4, D=128, o=3 * A, os=512):
        return lib.attn_rotary(None if table is None else ctypes.byref(table), x, xs, dtype, p, n, H, D, o, os, 0)

    assert call(n=0) == moe.MOE_OK
    assert call(n=-1) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(table=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(x=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(p=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(H=0) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(xs=504) == moe.MOE_ERR_INVALID_ARGUMENT      # rows over one another
    assert call(os=511) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(xs=1 << 62) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(o=A, os=520) == moe.MOE_ERR_INVALID_ARGUMENT  # onto itself with another stride
    assert call(o=A + 64) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(o=2 * A - 64) == moe.MOE_ERR_INVALID_ARGUMENT  # over the positions
    assert call(D=96) == moe.MOE_ERR_UNSUPPORTED
    assert call(D=64) == moe.MOE_ERR_UNSUPPORTED             # less than is turned
    assert call(dtype=2) == moe.MOE_ERR_UNSUPPORTED
    assert call(H=65537, xs=1 << 24, os=1 << 24) == moe.MOE_ERR_UNSUPPORTED
    assert call(x=A + 8) == moe.MOE_ERR_MISALIGNED
    assert call(xs=516) == moe.MOE_ERR_MISALIGNED
    cache = moe.attn_cache(A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, 2, 100, 64, 2, 64, 8, 20, 0)
    args = (7 * A, 8 * A, None, 9 * A, None, None, 0, 3, 30, 12 * A, 1 << 20, 0)
    assert lib.attn_cache_append_rotary(ctypes.byref(cache), None, *args) == moe.MOE_ERR_INVALID_ARGUMENT
    assert lib.attn_cache_append_rotary(ctypes.byref(cache), ctypes.byref(table), *args) == moe.MOE_ERR_UNSUPPORTED
    assert lib.attn_cache_append_rotary(None, ctypes.byref(table), *args) == moe.MOE_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [dict(), dict(base=1e6), dict(stretch=8.0), dict(base=5e5, stretch=16.0, low_turns=1.0,
                                                                               high_turns=32.0, original_len=4096.0)])
def test_the_table_holds_the_rates(lib, kw):
    rot = moe.make_rotary(256, **kw)
    w = rates(256, **kw)
    turns = np.array(list(rot.struct.turns), np.float64) / 2.0 ** 64
    want = w / (2 * np.pi)
    np.testing.assert_allclose(turns, want - np.floor(want), rtol=1e-14, atol=2.0 ** -60)


def test_stretched_rates_keep_the_fast_pairs_and_slow_the_others():
    f = rates(64, 10000.0)
    w = rates(64, 10000.0, 4.0, 1.0, 32.0, 4096.0)
    t = 4096 * f / (2 * np.pi)
    np.testing.assert_array_equal(w[t >= 32], f[t >= 32])
    np.testing.assert_array_equal(w[t <= 1], f[t <= 1] / 4)
    mid = (t > 1) & (t < 32)
    assert mid.any() and (w[mid] < f[mid]).all() and (w[mid] > f[mid] / 4).all()
    np.testing.assert_array_equal(rates(64, 10000.0, 4.0), f / 4)


@pytest.mark.parametrize("inter", [False, True])
def test_rotations_add_up_and_keep_products(inter):
    r = np.random.default_rng(1)
    w = rates(32)
    q, k = r.normal(size=(1, 2, 64)), r.normal(size=(1, 2, 64))
    turn = lambda x, p: rotate(x, [p], w, inter)  # noqa: E731
    np.testing.assert_allclose(turn(turn(q, 700), 42), turn(q, 742), atol=1e-10)
    # a product depends on the distance alone
    np.testing.assert_allclose((turn(q, 1000) * turn(k, 990)).sum(-1), (turn(q, 10) * turn(k, 0)).sum(-1), atol=1e-10)
    np.testing.assert_array_equal(turn(q, 5)[..., 32:], q[..., 32:])


def test_the_oracles_codes_and_scales():
    assert nearest([448, 449, 1e9, -500, 0.0, 17, 19, 2.0 ** -10, 2.0 ** -9 * 1.5]).tolist() == \
        [448, 448, 448, -448, 0, 16, 20, 0, 2.0 ** -8]
    assert np.isnan(nearest([np.nan, np.inf])).all()
    assert [scale_of(x) for x in (448, 448.0001, 224, 224.1, 0.0, 2.0 ** -120)] == [1, 2, 0.5, 1, 2.0 ** -100, 2.0 ** -100]
    page = QPages(np.zeros((1, 2, 16, 1, 4)), np.zeros((1, 2, 16, 1, 4)), np.zeros((1, 2, 1)), np.zeros((1, 2, 1)),
                  np.zeros(2, int), np.full((1, 2), -1), np.zeros(1, int))
    page.append([(0, np.full((1, 1, 1, 4), 7.0), np.ones((1, 1, 1, 4)))])
    assert page.ks[0, 0, 0] == 2.0 ** -6 and (page.k[0, 0, 0] == 448).all()
    page.append([(0, np.full((1, 1, 1, 4), 30.0), np.ones((1, 1, 1, 4)))])          # the scale grows: 7 is 112 of it
    assert page.ks[0, 0, 0] == 2.0 ** -3 and (page.k[0, 0, 0] == 56).all() and (page.k[0, 0, 1] == 240).all()
    np.testing.assert_array_equal(page.values(0)[0][:, 0, 0], [7.0, 30.0])


def test_attention_oracle_closed_forms():
    v = np.arange(12.0).reshape(6, 1, 2)
    o, mass, most = attend(np.zeros((2, 1, 2)), np.ones((6, 1, 2)), v)
    np.testing.assert_allclose(o[:, 0], [v[:5, 0].mean(0), v[:, 0].mean(0)])
    np.testing.assert_allclose(mass, o)
    assert (most == 0).all()
    o, _, _ = attend(np.ones((3, 1, 2)), np.ones((2, 1, 2)), np.ones((2, 1, 2)))  # a row before position 0
    np.testing.assert_allclose(o[:, 0, 0], [0, 1, 1])


@pytest.mark.parametrize("name", ["rotary.cu", "rotary.cuh", "qcache.cu", "qcache.cuh", "qattend.cu", "qattend.cuh",
                                  "qdecode.cu", "attn_join.cuh"])
def test_early_kernels_read_by_ordinary_loads(name):
    # a kernel that starts before the one ahead has ended reads data that changes while it runs: none of it
    # may go the read-only way, which __ldg and __restrict__ pointers to const ask for
    text = open(os.path.join(os.path.dirname(moe.__file__), "csrc", name)).read()
    for word in ("__ldg", "ld.global.nc", "__restrict__"):
        assert word not in text, f"{name}: {word}"


def test_binding_knows_its_types():
    torch = pytest.importorskip("torch")
    f8 = torch.zeros(1, 2, 16, 1, 64, dtype=torch.float8_e4m3fn)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):  # a 16-bit pool
        moe.make_attn_qcache(f8.half(), f8.half(), torch.zeros(1, 2, 1), torch.zeros(1, 2, 1), i, i[None], i[:1], i[:1])
    with pytest.raises(moe.MoeError):
        moe.make_rotary(24)
    assert moe.make_rotary(64, interleaved=True).struct.interleaved == 1
