"""Attention over the 8-bit paged cache where the pages' V scales lie far apart.

Tolerance: that of tests/test_gpu_qcache.py, with what a row sees in the place of what the
sequence holds.  A weight times its V scale is cut relative to the largest such product that
the row sees, to half of e5m2's least step where that is 2^6 or more: 2^-17 of 2^6, 2^-23.  So, with
sums and maxima over the positions that the row sees,
  u |o| + sum p|v| (2^-10 + 2 (e^d (1 + 2^-20) - 1) + l 2^-21) + 2^-22 max (p s) sum |code|,
u half a step of the output's type (bf16 2^-8, fp16 2^-11 and at least 2^-25) and d the error of a score.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle.qcache import scale_of

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import bit_grouped_expert_gb300 as moe  # noqa: E402
from tests.test_gpu_qcache import Case, f64  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_grouped_expert_gb300 import build
    build.build()


def rescale(c, b, factors, pool="v"):
    """Multiply the scales of a sequence's pages by factors [pages]; the expected values follow."""
    scales, which = (c.vs, 1) if pool == "v" else (c.ks, 0)
    page, slot, old = c.k.shape[2], c.slots[b], list(c.old[c.slots[b]])
    pages = c.table[slot, :len(factors)].long()
    scales[c.layer, pages] *= torch.tensor(factors, dtype=torch.float64, device=scales.device)[:, None].float()
    codes, _ = old[which]
    old[which] = (codes, f64(scales)[c.layer, pages.cpu().numpy()][np.arange(len(codes)) // page])
    c.old[slot] = old


def limits(c, b, scale=0.0):
    """The expected rows of sequence b and how far they may be off."""
    lo, n, L = int(c.off[b]), c.counts[b], c.lens[b]
    u, sc = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[c.dtype], scale or c.D ** -0.5
    q, ((kc, ks), (vc, vs)) = f64(c.q[lo:lo + n]), c.old[c.slots[b]]
    G = c.Hq // kc.shape[1]
    o, lim = np.zeros(q.shape), np.zeros(q.shape)
    for i in range(n):
        sees = L - n + i + 1
        for h in range(c.Hq):
            k, v = kc[:sees, h // G] * ks[:sees, h // G, None], np.abs(vc[:sees, h // G])
            s = k @ q[i, h] * sc
            p = np.exp(s - s.max())
            ps = p / p.sum() * vs[:sees, h // G]
            d = (sc * 2.0 ** -10 * scale_of(np.abs(q[i, h]).max()) * np.abs(k).sum(-1).max() +
                 (np.abs(k) @ np.abs(q[i, h])).max() * sc * c.D * 2.0 ** -22)
            o[i, h] = ps @ vc[:sees, h // G]
            lim[i, h] = (u * np.abs(o[i, h]) + 2.0 ** -25 * (c.dtype == "fp16") + 2.0 ** -130 +
                         ps @ v * (2.0 ** -10 + 2 * (np.exp(d) * (1 + 2.0 ** -20) - 1) + sees * 2.0 ** -21) +
                         2.0 ** -22 * ps.max() * v.sum(0))
    return o, lim


def check(c, scale=0.0):
    torch.cuda.synchronize()
    assert int(c.status[0]) == 0
    for b, n in enumerate(c.counts):
        lo = int(c.off[b])
        o, lim = limits(c, b, scale)
        held = np.abs(o) < (60000 if c.dtype == "fp16" else 2.0 ** 127)  # by the output's type
        err = np.where(held, np.abs(f64(c.o[lo:lo + n]) - o), 0.0)
        assert (err <= lim).all(), (b, float((err / lim).max()))


# Few rows a unit and many, one sequence cut over the CTAs and units that are not; the last token alone in its page.
KINDS = [(4, 2, 64, "fp16", [3009], [2]), (4, 2, 64, "fp16", [113] * 30, [2] * 30), (8, 1, 256, "bf16", [3009], [5]),
         (8, 2, 128, "bf16", [49] * 40, [3] * 40), (16, 2, 256, "fp16", [113, 2001], [2, 16]), (8, 1, 128, "bf16", [1505], [2])]


@pytest.mark.parametrize("factor", [2.0 ** 13, 2.0 ** 20, 2.0 ** 30, 2.0 ** 100])
@pytest.mark.parametrize("Hq,Hkv,D,dtype,lens,counts", KINDS)
def test_a_scale_behind_a_row_cannot_change_it(Hq, Hkv, D, dtype, lens, counts, factor):
    c = Case(40, lens, counts, Hq, Hkv, D, 16, dtype)
    a = c.run().clone()
    check(c)
    before = np.ones(int(c.off[-1]), bool)
    before[c.off[1:] - 1] = False  # all rows but each sequence's last
    for b, L in enumerate(lens):
        rescale(c, b, [1.0] * (-(-L // 16) - 1) + [factor])
    r = c.run().clone()
    torch.cuda.synchronize()
    assert torch.equal(a[before], r[before])
    check(c)
    # bits of any kind where nobody looks: the rows that do not see the page stay as they are
    for bad in (float("inf"), float("nan"), -1.0):
        for b, L in enumerate(lens):
            c.vs[0, c.table[b, (L - 1) // 16].long()] = bad
            c.ks[0, c.table[b, (L - 1) // 16].long()] = bad
        r = c.run().clone()
        torch.cuda.synchronize()
        assert torch.equal(a[before], r[before])


@pytest.mark.parametrize("factor,weight", [(2.0 ** 13, 30), (2.0 ** 20, 60), (2.0 ** 30, 90), (2.0 ** 30, 32), (2.0 ** 60, 100)])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("Hq,D,rows", [(4, 64, 1), (8, 256, 2), (8, 128, 5), (16, 256, 4)])
def test_a_large_scale_seen_with_next_to_no_weight(Hq, D, rows, first, factor, weight):
    # page 0 or the one before the rows has scores `weight` binary orders below the others, and a V scale far above
    for L in (300, 5000):
        c = Case(41, [L], [rows], Hq, 1, D, 16)
        c.q[:] = 1.0
        at = 0 if first else (L - rows) // 16 - 1
        codes, scales = c.old[0][0]
        codes[:] = 0.0
        codes[16 * at:16 * at + 16] = -2.0
        pages = c.table[0].long()
        c.k.view(torch.uint8)[0, pages] = 0
        c.k.view(torch.uint8)[0, pages[at]] = 0xC0      # -2
        c.ks[0, pages] = 0.25
        scales[:] = 0.25
        rescale(c, 0, [factor if j == at else 1.0 for j in range(-(-L // 16))])
        scale = weight * np.log(2.0) / (0.5 * D)
        c.run(scale)
        check(c, scale)


@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("low,high", [(-30, 10), (-90, 60)])
@pytest.mark.parametrize("Hq,D,rows,dtype", [(8, 128, 1, "bf16"), (4, 64, 2, "bf16"), (8, 256, 3, "bf16"), (16, 256, 8, "bf16"),
                                             (16, 64, 8, "fp16")])
def test_scales_that_rise_and_fall(Hq, D, rows, dtype, low, high, up):
    for L in (400, 2000):
        c = Case(42, [L], [rows], Hq, 1, D, 16, dtype)
        f = 2.0 ** np.linspace(low, high if dtype == "bf16" else min(high, 10), -(-L // 16))
        rescale(c, 0, f if up else f[::-1].copy())
        rescale(c, 0, np.linspace(0.5, 4.0, len(f)), "k")
        c.run()
        check(c)


@pytest.mark.parametrize("Hq,D,rows", [(8, 128, 1), (4, 64, 2), (16, 256, 4), (16, 128, 8)])
def test_most_weight_on_a_page_of_zeros(Hq, D, rows):
    # as an append leaves one: codes 0, the least scale; what is left of the weight is all that counts
    for L in (200, 5000):
        c = Case(43, [L], [rows], Hq, 1, D, 16)
        c.q[:] = 1.0
        pages = c.table[0].long()
        c.v.view(torch.uint8)[0, pages[0]] = 0
        c.old[0][1][0][:16] = 0.0
        c.vs[0, pages[0]] = 2.0 ** -100
        c.old[0][1][1][:16] = 2.0 ** -100
        c.k.view(torch.uint8)[0, pages] = 0
        c.k.view(torch.uint8)[0, pages[0]] = 0x38       # 1
        c.old[0][0][0][:] = 0.0
        c.old[0][0][0][:16] = 1.0
        c.ks[0, pages] = 1.0
        c.old[0][0][1][:] = 1.0
        for orders in (20, 40):
            c.run(orders * np.log(2.0) / D)
            check(c, orders * np.log(2.0) / D)
