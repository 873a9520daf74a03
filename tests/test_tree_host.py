"""Host checks of the paged-cache, tree-attention and verification entry
points: every call here is refused on the host, or has nothing to do, before
anything is enqueued (safe with or without a GPU)."""
from __future__ import annotations

import ctypes

import pytest

import bit_grouped_expert_gb300 as moe


@pytest.fixture(scope="module")
def lib():
    from bit_grouped_expert_gb300 import build
    build.build()
    return moe.lib()


A = 0x10000000  # fake, aligned device addresses


def _cache(**kw):
    d = dict(k_d=A, v_d=2 * A, refs_d=3 * A, table_d=4 * A, lens_d=5 * A, status_d=6 * A, n_layers=2, n_pages=100,
             page_size=64, n_kv_heads=2, head_dim=256, n_slots=8, max_pages=20, dtype=moe.MOE_BF16)
    d.update(kw)
    return moe.attn_cache(**d)


def _ref(c):
    return ctypes.byref(c) if c is not None else None


BAD_CACHES = [(dict(k_d=None), moe.MOE_ERR_INVALID_ARGUMENT), (dict(status_d=None), moe.MOE_ERR_INVALID_ARGUMENT),
              (dict(n_pages=0), moe.MOE_ERR_INVALID_ARGUMENT), (dict(n_slots=-1), moe.MOE_ERR_INVALID_ARGUMENT),
              (dict(page_size=48), moe.MOE_ERR_UNSUPPORTED), (dict(page_size=8), moe.MOE_ERR_UNSUPPORTED),
              (dict(page_size=512), moe.MOE_ERR_UNSUPPORTED), (dict(head_dim=96), moe.MOE_ERR_UNSUPPORTED),
              (dict(dtype=2), moe.MOE_ERR_UNSUPPORTED), (dict(n_kv_heads=257), moe.MOE_ERR_UNSUPPORTED),
              (dict(n_pages=1 << 25), moe.MOE_ERR_UNSUPPORTED), (dict(max_pages=1 << 25), moe.MOE_ERR_UNSUPPORTED),
              (dict(max_pages=(1 << 24) + 1), moe.MOE_ERR_UNSUPPORTED),
              (dict(v_d=A + 8), moe.MOE_ERR_MISALIGNED), (dict(table_d=A + 4), moe.MOE_ERR_MISALIGNED)]


def _append(lib, c=None, B=3, rows=30, ws=None, stride=4, null_cache=False, **kw):
    c = _cache() if c is None else c
    a = {**dict(k=7 * A, v=8 * A, slots=None, off=9 * A, keep=10 * A, path=11 * A, ws=12 * A), **kw}
    need = lib.attn_cache_append_workspace_bytes(_ref(c), B, rows) if ws is None else ws
    return lib.attn_cache_append(None if null_cache else _ref(c), a["k"], a["v"], a["slots"], a["off"], a["keep"],
                                 a["path"], stride, B, rows, a["ws"], need, 0)


@pytest.mark.parametrize("change,want", BAD_CACHES)
def test_bad_caches_are_refused_by_every_entry_point(lib, change, want):
    c = _cache(**change)
    assert _append(lib, c, ws=1 << 20) == want
    assert lib.attn_cache_fork(_ref(c), A, A, 2, A, 1 << 20, 0) == want
    assert lib.attn_cache_trim(_ref(c), A, A, 2, 0) == want
    assert lib.attn_tree(_ref(c), 0, A, A, A, None, A, A, 1, 4, 4, 16, ctypes.c_float(0), A, 1 << 30, A, 0) == want
    assert lib.attn_cache_append_workspace_bytes(_ref(c), 1, 1) == 0
    assert lib.attn_cache_fork_workspace_bytes(_ref(c), 1) == 0
    assert lib.attn_tree_workspace_bytes(_ref(c), 1, 1, 1, 16) == 0


def test_append_host_checks(lib):
    assert _append(lib, null_cache=True) == moe.MOE_ERR_INVALID_ARGUMENT
    assert _append(lib, B=0) == moe.MOE_OK
    assert _append(lib, B=-1) == moe.MOE_ERR_INVALID_ARGUMENT
    assert _append(lib, rows=-1) == moe.MOE_ERR_INVALID_ARGUMENT
    assert _append(lib, k=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert _append(lib, off=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert _append(lib, keep=None) == moe.MOE_ERR_INVALID_ARGUMENT  # a path without its lengths
    assert _append(lib, stride=0) == moe.MOE_ERR_INVALID_ARGUMENT
    assert _append(lib, B=1025, ws=1 << 30) == moe.MOE_ERR_UNSUPPORTED
    assert _append(lib, v=A + 2) == moe.MOE_ERR_MISALIGNED
    assert _append(lib, path=A + 4) == moe.MOE_ERR_MISALIGNED
    pool = 2 * 100 * 64 * 512 * 2  # bytes of K
    assert _append(lib, k=A + pool - 16) == moe.MOE_ERR_INVALID_ARGUMENT  # rows inside the pool
    assert _append(lib, v=2 * A) == moe.MOE_ERR_INVALID_ARGUMENT
    need = lib.attn_cache_append_workspace_bytes(_ref(_cache()), 3, 30)
    assert need > 0 and _append(lib, ws=need - 1) == moe.MOE_ERR_WORKSPACE_TOO_SMALL


def test_fork_and_trim_host_checks(lib):
    c = _cache()
    need = lib.attn_cache_fork_workspace_bytes(_ref(c), 4)

    def fork(src=A, dst=2 * A, n=4, ws=3 * A, nb=need):
        return lib.attn_cache_fork(_ref(c), src, dst, n, ws, nb, 0)

    assert fork(n=0, src=None) == moe.MOE_OK
    assert fork(n=-1) == moe.MOE_ERR_INVALID_ARGUMENT
    assert fork(dst=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert fork(ws=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert fork(n=1025, nb=1 << 20) == moe.MOE_ERR_UNSUPPORTED
    assert fork(src=A + 4) == moe.MOE_ERR_MISALIGNED
    assert fork(nb=need - 1) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    assert lib.attn_cache_fork(None, A, A, 1, A, 1 << 20, 0) == moe.MOE_ERR_INVALID_ARGUMENT
    assert lib.attn_cache_trim(_ref(c), None, None, 0, 0) == moe.MOE_OK
    assert lib.attn_cache_trim(_ref(c), None, None, 1, 0) == moe.MOE_ERR_INVALID_ARGUMENT
    assert lib.attn_cache_trim(_ref(c), None, A, -1, 0) == moe.MOE_ERR_INVALID_ARGUMENT
    assert lib.attn_cache_trim(_ref(c), None, A, 1025, 0) == moe.MOE_ERR_UNSUPPORTED
    assert lib.attn_cache_trim(_ref(c), A + 4, A, 1, 0) == moe.MOE_ERR_MISALIGNED


def test_tree_host_checks(lib):
    def call(c=None, layer=0, B=2, n=10, mx=8, Hq=16, scale=0.0, nb=None, **kw):
        c = _cache() if c is None else c
        a = {**dict(q=7 * A, k=8 * A, v=9 * A, slots=None, off=10 * A, par=11 * A, ws=12 * A, o=13 * A), **kw}
        need = lib.attn_tree_workspace_bytes(_ref(c), B, n, mx, Hq) if nb is None else nb
        return lib.attn_tree(_ref(c), layer, a["q"], a["k"], a["v"], a["slots"], a["off"], a["par"], B, n, mx, Hq,
                             ctypes.c_float(scale), a["ws"], need, a["o"], 0)

    assert call(B=0) == moe.MOE_OK
    assert call(n=0, q=None) == moe.MOE_OK
    assert call(layer=2) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(layer=-1) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(B=-1) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(mx=0) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(Hq=0) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(scale=-0.5) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(scale=float("nan")) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(scale=float("inf")) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(par=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(o=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(Hq=15, nb=1 << 30) == moe.MOE_ERR_UNSUPPORTED
    assert call(Hq=258, nb=1 << 30) == moe.MOE_ERR_UNSUPPORTED  # 129 query heads per KV head
    assert call(mx=257, nb=1 << 30) == moe.MOE_ERR_UNSUPPORTED
    assert call(B=1025, nb=1 << 30) == moe.MOE_ERR_UNSUPPORTED
    assert call(q=7 * A + 2) == moe.MOE_ERR_MISALIGNED
    for x in (7, 8, 9):  # the output over an input, or inside the pool
        assert call(o=x * A + 16) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(o=A + 4096) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(slots=A + 4) == moe.MOE_ERR_MISALIGNED
    need = lib.attn_tree_workspace_bytes(_ref(_cache()), 2, 10, 8, 16)
    assert need > 0 and call(nb=need - 1) == moe.MOE_ERR_WORKSPACE_TOO_SMALL


def test_verify_host_checks(lib):
    def call(B=2, n=10, V=100, stride=8, **kw):
        a = {**dict(p=A, q=2 * A, tok=3 * A, par=4 * A, off=5 * A, ua=6 * A, us=7 * A, path=8 * A, np=9 * A, nx=10 * A,
                    st=11 * A), **kw}
        return lib.moe_draft_verify(a["p"], a["q"], a["tok"], a["par"], a["off"], a["ua"], a["us"], B, n, V, a["path"],
                                    stride, a["np"], a["nx"], a["st"], 0)

    assert call(B=0, p=None) == moe.MOE_OK
    assert call(B=-1) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(V=0) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(stride=0) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(p=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(us=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(st=None) == moe.MOE_ERR_INVALID_ARGUMENT
    assert call(V=(1 << 20) + 1) == moe.MOE_ERR_UNSUPPORTED
    assert call(stride=1025) == moe.MOE_ERR_UNSUPPORTED
    assert call(B=65536) == moe.MOE_ERR_UNSUPPORTED
    assert call(q=A + 4) == moe.MOE_ERR_MISALIGNED
    assert call(path=A + 8) == moe.MOE_ERR_MISALIGNED


def test_status_text():
    assert moe.status_str(moe.MOE_ERR_OUT_OF_PAGES) == "too few free cache pages"


@pytest.mark.parametrize("name", ["tree.cu", "draft.cu", "cache.cu", "cache.cuh"])
def test_early_kernels_read_by_ordinary_loads(name):
    # a kernel that starts before the one ahead has ended reads data that changes while it runs: none of it
    # may go the read-only way, which __ldg and __restrict__ pointers to const ask for
    import os
    src = os.path.join(os.path.dirname(moe.__file__), "csrc", name)
    text = open(src).read()
    for word in ("__ldg", "ld.global.nc", "__restrict__"):
        assert word not in text, f"{name}: {word}"
