"""The 8-bit paged cache at its larger sizes: pools whose layers pass 2^31 bytes, and attention of whole chunks of a
prompt.  Tolerances: those of tests/test_gpu_qcache_range.py."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import bit_grouped_expert_gb300 as moe  # noqa: E402
from tests.test_gpu_qcache import DEV, F8, Case, Twin, i32  # noqa: E402
from tests.test_gpu_qcache_range import check  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_grouped_expert_gb300 import build
    build.build()


PAGES = 17000  # of 256 rows of 2 heads of 256: a layer of 2.2 GB


def big_pools(layers, dtype=F8):
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 20 GB")
    return [torch.empty(layers, PAGES, 256, 2, 256, dtype=torch.uint8 if dtype is F8 else dtype, device=DEV).view(dtype)
            for _ in "kv"]


@pytest.mark.parametrize("rows", [2, 40])  # the kernel for few rows, and whole matrices
@pytest.mark.parametrize("layer", [0, 1])
def test_attention_in_a_layer_of_more_than_31_bits(layer, rows):
    c = Case(50, [500, 277], [rows, rows], 4, 2, 256, 256)
    pools = big_pools(layer + 1)
    scales = [torch.full((layer + 1, PAGES, 2), float("nan"), device=DEV) for _ in "kv"]
    move = {int(p): PAGES - 1 - i for i, p in enumerate(c.table[c.table >= 0].tolist())}
    for big, small, s, ss in zip(pools, (c.k, c.v), scales, (c.ks, c.vs)):
        for a, b in move.items():
            big.view(torch.uint8)[layer, b] = small.view(torch.uint8)[0, a]
            s[layer, b] = ss[0, a]
    table = i32([[move.get(p, -1) for p in row] for row in c.table.tolist()])
    cache = moe.make_attn_qcache(*pools, *scales, i32([1] * PAGES), table, c.slot_lens, c.status)

    def run():
        moe.attn_qcache_attend(cache, layer, c.q, i32(c.off.tolist()), 2, c.max_rows, c.ws, c.o)
        return c.o

    a = run().clone()
    check(c)
    # a code NaN that only the last row of a sequence sees: looked up once more in the pool
    for b, L in enumerate(c.lens):
        pools[1].view(torch.uint8)[layer, int(table[b, (L - 1) // 256]), (L - 1) % 256, 1, 77] = 0x7F
    r = run()
    torch.cuda.synchronize()
    want = torch.zeros_like(r, dtype=torch.bool)
    want[[rows - 1, 2 * rows - 1], 2:, 77] = True
    assert torch.equal(r.isnan(), want) and torch.equal(a[~want], r[~want])


@pytest.mark.parametrize("turned", [False, True])
def test_appends_and_forks_beyond_31_bits(turned):
    # the same calls on a small cache and on one whose only free pages are the last: equal pages
    t = Twin(256, 2, 256, "bf16", pages=8, slots=4, max_pages=3, layers=2)
    pools = big_pools(2)
    scales = [torch.full((2, PAGES, 2), 4.0, device=DEV) for _ in "kv"]
    refs, table, lens = i32([1] * (PAGES - 8) + [0] * 8), torch.full((4, 3), -1, dtype=torch.int32, device=DEV), i32([0] * 4)
    big = moe.make_attn_qcache(*pools, *scales, refs, table, lens, t.status)
    rot = moe.make_rotary(64) if turned else None
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)
    for gain, counts, slots in ((1.0, [300, 5], [0, 1]), (9.0, [20, 1], [0, 1]), (50.0, [3, 2, 7], [2, 0, 1])):
        n = sum(counts)
        rows = [t.normal(2, n, 2, 256) * gain for _ in "kv"]
        off = i32([sum(counts[:i]) for i in range(len(counts) + 1)])
        for cache in (t.cache, big):
            moe.attn_qcache_append(cache, rot, *rows, off, len(counts), ws, slots=i32(slots))
        if gain == 9.0:
            for cache in (t.cache, big):
                moe.attn_qcache_fork(cache, i32([0]), i32([2]), 1, ws)  # (the next append copies its last page)
    torch.cuda.synchronize()
    assert int(t.status[0]) == 0 and torch.equal(t.lens, lens)
    used = t.table >= 0
    assert torch.equal(used, table >= 0) and int(table[used].min()) >= PAGES - 8
    small, far = t.table[used].long(), table[used].long()
    for a, b in ((t.ks, scales[0]), (t.vs, scales[1])):
        assert torch.equal(a[:, small], b[:, far])
    for slot, L in enumerate(lens.tolist()):
        for p in range(-(-L // 256)):
            n = min(256, L - 256 * p)
            for a, b in ((t.k, pools[0]), (t.v, pools[1])):
                assert torch.equal(a.view(torch.uint8)[:, int(t.table[slot, p]), :n],
                                   b.view(torch.uint8)[:, int(table[slot, p]), :n])


def test_turned_appends_beyond_31_bits_in_16_bits():
    pools = big_pools(1, torch.bfloat16)
    small = [torch.zeros(1, 4, 256, 2, 256, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    rot, status = moe.make_rotary(128, interleaved=True), i32([0] * 4)
    tables, lens = [torch.full((2, 2), -1, dtype=torch.int32, device=DEV) for _ in "ab"], [i32([0, 0]) for _ in "ab"]
    caches = [moe.make_attn_cache(*p, i32(r), t, l, status) for p, r, t, l in
              ((small, [0] * 4, tables[0], lens[0]), (pools, [1] * (PAGES - 4) + [0] * 4, tables[1], lens[1]))]
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)
    for n in (270, 7):
        rows = [torch.empty(1, n, 2, 256, dtype=torch.bfloat16, device=DEV).normal_() for _ in "kv"]
        for cache in caches:
            moe.attn_cache_append_rotary(cache, rot, *rows, i32([0, n - 3, n]), 2, ws)
    torch.cuda.synchronize()
    assert int(status[0]) == 0 and lens[0].tolist() == lens[1].tolist() == [271, 6]
    for slot, p, n in ((0, 0, 256), (0, 1, 15), (1, 0, 6)):
        for a, b in zip(small, pools):
            assert torch.equal(a[:, int(tables[0][slot, p]), :n], b[:, int(tables[1][slot, p]), :n])


# A prompt's chunk: 500 rows to 2,500 of a sequence, one token a row tile (128 heads on one) and whole tiles of tokens.
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype,lens,counts", [
    (2, 1, 64, 64, "bf16", [2600], [2500]), (4, 2, 128, 16, "fp16", [900, 1400], [900, 650]),
    (8, 1, 256, 256, "bf16", [1300, 20], [520, 20]), (128, 1, 64, 32, "bf16", [400], [300]),
    (5, 1, 128, 128, "bf16", [1000], [1001])])
def test_chunks_of_a_prompt(Hq, Hkv, D, page, dtype, lens, counts):
    c = Case(51, lens, counts, Hq, Hkv, D, page, dtype, behind=2)
    c.run()
    if counts[0] > lens[0]:  # the row in front of the sequence sees nothing
        torch.cuda.synchronize()
        assert not c.o[0].any()
        c.counts, c.off, c.q, c.o = [counts[0] - 1], c.off - [0, 1], c.q[1:], c.o[1:]
    check(c)
    assert (c.o[int(c.off[-1]):] == 7.0).all()
