"""GPU: the paged cache with a scale per block of tokens and head.  What is written has to equal the
fp64 oracle bit for bit; attention has to lie within a bound of its own roundings:

  fp32 sums of D products, any order:      (D + 8) 2^-23 of the sum of their magnitudes,
  twice in the weights (own and largest):  e = 2 ((D + 8) 2^-23 Smax + 2^-21) with the exponential's
                                           own 2^-22 and the scale's roundings,
  sums over n keys:                        (n + 16) 2^-23,
  the weights' rounding to bf16:           2^-8 (bf16 rows) or, held in three terms, 2^-22,
  the result's rounding:                   2^-8 or 2^-24 of itself,
the first three and the weights' relative to sum w |v|."""
import numpy as np
import pytest

from oracle import blocks, lowp

from block_util import DT, BlockCache, ints, scattered, starts_of
from gpu_util import host, need_gpu, say, torch

pytestmark = pytest.mark.gpu


def _same_cache(c, want):
    codes, scales = c.host()
    if c.fmt == "e4m3":  # a NaN's sign stands for nothing
        codes, want = np.where(codes == 255, 127, codes), (np.where(want[0] == 255, 127, want[0]), want[1])
    assert np.array_equal(codes, want[0])
    assert np.array_equal(scales, want[1])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("lens,news,page,block,heads,dim,order,dt", [
    ([1], [1], 1, 1, 1, 16, "phd", "bf16"),
    ([5, 17, 32, 1, 40], [1, 1, 1, 1, 1], 16, 16, 3, 64, "phd", "bf16"),
    ([5, 17, 33, 3, 0, 48], [5, 16, 3, 0, 0, 20], 16, 8, 2, 128, "hpd", "f32"),
    ([150, 99, 101], [150, 7, 2], 100, 20, 5, 80, "phd", "bf16"),
    ([300, 64, 70], [300, 64, 1], 64, 64, 2, 256, "hpd", "bf16"),
    ([700], [650], 256, 256, 1, 128, "phd", "f32"),
    ([9, 3], [12, 3], 4, 2, 2, 32, "phd", "f32"),  # more rows than the sequence is long
])
def test_write(fmt, lens, news, page, block, heads, dim, order, dt):
    q = need_gpu()
    rng = np.random.default_rng(sum(lens) + dim)
    table, pages = scattered(rng, lens, page)
    kb, vb = (BlockCache(q, rng, pages, page, block, heads, dim, fmt, order) for _ in range(2))
    T = sum(news) + 2  # two rows of padding
    kv = torch.from_numpy(rng.standard_t(4, size=(T, 3 * heads, dim)) * 3).to(DT[dt])
    kv[0, heads] = 0.0
    if T > 4:
        kv[2] *= 1e-30
        kv[4] *= 1e6
    K, V = kv[:, heads:2 * heads], kv[:, 2 * heads:]
    want = [c.host() for c in (kb, vb)]
    st = starts_of(news)
    for w, x in zip(want, (K, V)):
        blocks.write(*w, fmt, x.double().numpy(), table, lens, st)
    d = kv.cuda()
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    say("block write", fmt, lens, news, page, block, heads, dim, order, dt)
    q.kv_block_write(d[:, heads:2 * heads], d[:, 2 * heads:], kb.h, vb.h, ints(table), ints(lens), ints(st), info=info)
    torch.cuda.synchronize()
    assert int(info) == 0
    _same_cache(kb, want[0])
    _same_cache(vb, want[1])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_blocks_grow_row_by_row(fmt):
    """Decode steps into one block, each row larger than the ones before, then rows taken back."""
    q = need_gpu()
    rng = np.random.default_rng(5)
    heads, dim, page = 2, 64, 16
    c = BlockCache(q, rng, 3, page, page, heads, dim, fmt)
    want = c.host()
    table = [[2, 0]]
    say("block growth", fmt)
    n = 0
    for step in range(24):
        if step == 17:
            n -= 6  # refused drafts: their places are written again
        n += 1
        x = torch.from_numpy(rng.normal(size=(1, heads, dim)) * 1.7 ** (step % 11)).to(torch.bfloat16)
        blocks.write(*want, fmt, x.double().numpy(), table, [n], [0, 1])
        q.kv_block_write(x.cuda(), None, c.h, None, ints(table), ints([n]), ints([0, 1]))
        _same_cache(c, want)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_write_non_finite_and_unwritten_scales(fmt):
    q = need_gpu()
    rng = np.random.default_rng(6)
    c = BlockCache(q, rng, 2, 8, 8, 1, 32, fmt)
    c.scales[0] = float("nan")  # a block that was never written, rows added to it
    c.scales[1] = 0.0
    want = c.host()
    x = torch.from_numpy(rng.normal(size=(5, 1, 32))).float()
    x[1, 0, 3], x[2, 0, 4], x[3, 0, 5] = float("nan"), float("inf"), float("-inf")
    x[4] = float("inf")
    table = [[0], [1]]
    blocks.write(*want, fmt, x.double().numpy(), table, [6, 7], [0, 3, 5])
    say("block write non-finite", fmt)
    q.kv_block_write(x.cuda(), None, c.h, None, ints(table), ints([6, 7]), ints([0, 3, 5]))
    _same_cache(c, want)


def test_write_bad_pages():
    """Pages that are none, positions past the table: left out, reported, everything else written."""
    q = need_gpu()
    rng = np.random.default_rng(7)
    c = BlockCache(q, rng, 4, 4, 4, 2, 16, "e4m3")
    want = c.host()
    table, lens, news = [[1, -1], [4, 2], [0, 3]], [7, 8, 11], [7, 8, 11]
    x = torch.from_numpy(rng.normal(size=(sum(news), 2, 16))).float()
    assert blocks.write(*want, "e4m3", x.double().numpy(), table, lens, starts_of(news))
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    say("block write bad pages")
    q.kv_block_write(x.cuda(), None, c.h, None, ints(table), ints(lens), ints(starts_of(news)), info=info)
    _same_cache(c, want)
    assert int(info) == 1


def _attend(q, rng, lens, news, page, block, heads, group, dim, fmt, dt, order="phd", causal=True, window=0,
            pad=0, scale=None, spoil=True, qscale=1.0, table=None):
    """One call against the oracle; returns (out, lse)."""
    if table is None:
        table, pages = scattered(rng, lens, page)
    else:
        pages = 1 + max(max(r) for r in table)
    kb, vb = (BlockCache(q, rng, pages, page, block, heads, dim, fmt, order) for _ in range(2))
    T, HQ = sum(news) + pad, heads * group
    x = torch.from_numpy(rng.normal(size=(T, HQ + 2, dim)) * qscale).to(DT[dt])
    kw = dict(causal=causal, window=window, scale=scale)
    ref, rlse, mag, smax = blocks.attention(x[:, 1:HQ + 1].double().numpy(), *kb.host(), *vb.host(), fmt, table, lens,
                                            starts_of(news), **kw)
    if spoil:  # places that no row sees hold what is no number
        used = np.zeros((pages, page), bool)
        for r, n in zip(table, lens):
            for p in range(n):
                if p // page < len(r) and r[p // page] >= 0:
                    used[r[p // page], p % page] = True
        free = torch.from_numpy(~used).cuda()
        blk = torch.from_numpy(~used.reshape(pages, -1, block).any(2)).cuda()
        for c in (kb, vb):
            c.codes[free] = 0x7F
            c.scales[blk] = float("nan")
    xd = x.cuda()
    out = torch.full((T, HQ, dim + 8), 7.0, dtype=DT[dt], device="cuda")
    lse = torch.full((T, HQ), 7.0, device="cuda")
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    say("attend", lens, news, page, block, heads, group, dim, fmt, dt, order, causal, window)
    q.kv_block_attention(xd[:, 1:HQ + 1], kb.h, vb.h, ints(table), ints(lens), ints(starts_of(news)), out[..., :dim],
                         lse=lse, info=info, **kw)
    torch.cuda.synchronize()
    got, glse = host(out[..., :dim].double()), host(lse.double())
    n = sum(news)
    assert np.all(got[n:] == 7) and np.all(glse[n:] == 7)  # rows behind the last sequence
    assert bool((out[..., dim:] == 7).all())
    ref, rlse, mag, smax, got, glse = ref[:n], rlse[:n], mag[:n], smax[:n], got[:n], glse[:n]
    assert np.array_equal(np.isneginf(glse), np.isneginf(rlse))
    keys = max(list(lens) + [1])
    e = 2 * ((dim + 8) * 2.0 ** -23 * smax + 2.0 ** -21) + (keys + 16) * 2.0 ** -23
    w, half = (2.0 ** -8, 2.0 ** -8) if dt == "bf16" else (2.0 ** -22, 2.0 ** -24)
    # (a weight below fp32's smallest normal number 2^-126 may be lost: times a value, at most 448 * 0.03 < 2^4)
    tol = half * np.abs(ref) + (1 + half) * (w * (1 + e) + e)[..., None] * mag + keys * 2.0 ** -122
    assert np.all(np.abs(got - ref) <= tol), np.nanmax((np.abs(got - ref) - tol))
    real = np.isfinite(rlse)
    glse, rlse = np.where(real, glse, 0.0), np.where(real, rlse, 0.0)
    # the logarithm's own roundings: of the maximum's product, of the logarithm, of their sum
    assert np.all(np.abs(glse - rlse)[real] <= e[real] + 2.0 ** -22 * (2 + np.abs(rlse[real]) + smax[real]))
    return int(info)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("lens,news,page,block,heads,group,dim,dt,kw", [
    ([1], [1], 1, 1, 1, 1, 16, "bf16", {}),
    ([300, 17, 1, 64], [1, 1, 1, 1], 16, 16, 2, 4, 128, "bf16", {"pad": 2}),
    ([301, 16, 31, 33], [1, 1, 1, 1], 16, 16, 1, 8, 64, "f32", {}),
    ([40, 0, 5, 90], [3, 0, 5, 2], 32, 16, 2, 2, 96, "bf16", {"order": "hpd"}),
    ([205, 99, 7], [5, 4, 7], 100, 20, 2, 2, 80, "f32", {"window": 50, "order": "hpd"}),
    ([130, 50], [130, 20], 64, 64, 2, 1, 128, "bf16", {}),
    ([77, 80], [77, 33], 16, 1, 1, 3, 256, "bf16", {"window": 16}),
    ([50, 60], [4, 60], 20, 5, 1, 2, 192, "f32", {"causal": False}),
    ([200, 30], [9, 30], 128, 128, 1, 5, 48, "bf16", {"causal": False, "scale": 0.5}),
    ([3, 9], [6, 12], 4, 4, 2, 2, 32, "bf16", {}),  # rows in front of position 0 see nothing
    ([70], [70], 16, 16, 1, 2, 64, "bf16", {"window": 1}),
    ([3000, 10, 1500], [1, 1, 2], 64, 32, 1, 4, 64, "bf16", {}),  # splits
    ([2500], [3], 7, 7, 1, 2, 32, "f32", {}),
    ([1100, 900], [20, 20], 16, 16, 1, 4, 64, "bf16", {"window": 300}),
])
def test_attention(fmt, lens, news, page, block, heads, group, dim, dt, kw):
    q = need_gpu()
    rng = np.random.default_rng(sum(lens) * 7 + dim)
    assert _attend(q, rng, lens, news, page, block, heads, group, dim, fmt, dt, **kw) == 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 6])
def test_attention_bad_pages(dt, page):
    """Keys whose page is none are not there."""
    q = need_gpu()
    rng = np.random.default_rng(3)
    table = [[0, -1, 2, 3], [-1, -1, -1, -1], [5, 1, 1000, 4]]
    lens = [4 * page, 2 * page, 5 * page]  # the last one is longer than its row
    table[2][2] = 6  # one past the last page
    pages = 6
    kb, vb = (BlockCache(q, rng, pages, page, 2 if page == 6 else 16, 1, 32, "e4m3") for _ in range(2))
    x = torch.from_numpy(rng.normal(size=(3, 2, 32))).to(DT[dt])
    ref, rlse, mag, smax = blocks.attention(x.double().numpy(), *kb.host(), *vb.host(), "e4m3", table, lens, [0, 1, 2, 3])
    out, lse = torch.empty((3, 2, 32), dtype=DT[dt], device="cuda"), torch.empty((3, 2), device="cuda")
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    say("attend bad pages", dt, page)
    q.kv_block_attention(x.cuda(), kb.h, vb.h, ints(table), ints(lens), ints([0, 1, 2, 3]), out, lse=lse, info=info)
    assert int(info) == 1
    half = 2.0 ** -8 if dt == "bf16" else 2.0 ** -20
    assert np.all(host(out.double())[1] == 0) and np.all(np.isneginf(host(lse)[1]))
    assert np.all(np.abs(host(out.double()) - ref) <= half * np.abs(ref) + 1.1 * (half + 2.0 ** -14) * mag)


@pytest.mark.parametrize("dt,news", [("bf16", 6), ("bf16", 40), ("f32", 6)])
@pytest.mark.parametrize("page", [16, 10])
def test_attention_nan_reaches_only_rows_that_see_it(dt, news, page):
    """A NaN among the keys or values of position p: rows from p on are NaN (of the values: in its
    column), the others are as if it were not there."""
    q = need_gpu()
    n = 50
    for side in ("key", "value"):
        rng = np.random.default_rng(8)
        table, pages = scattered(rng, [n], page)
        kb, vb = (BlockCache(q, rng, pages, page, 2 if page == 10 else 16, 1, 64, "e4m3") for _ in range(2))
        x = torch.from_numpy(rng.normal(size=(news, 2, 64))).to(DT[dt]).cuda()
        args = (ints(table), ints([n]), ints([0, news]))
        clean = torch.empty((news, 2, 64), dtype=DT[dt], device="cuda")
        q.kv_block_attention(x, kb.h, vb.h, *args, clean)
        p = n - 3
        c = kb if side == "key" else vb
        c.codes[table[0][p // page], p % page, 0, 21] = 0xFF
        out = torch.empty_like(clean)
        say("attend nan", dt, news, page, side)
        q.kv_block_attention(x, kb.h, vb.h, *args, out)
        want = torch.zeros((news, 2, 64), dtype=torch.bool, device="cuda")
        if side == "key":
            want[news - 3:] = True
        else:
            want[news - 3:, :, 21] = True
        assert torch.equal(torch.isnan(out), want), side
        assert torch.equal(out[~want], clean[~want])


def test_attention_extreme_scores():
    """Scores of many thousands, of one sign or the other: a running maximum, no overflow."""
    q = need_gpu()
    rng = np.random.default_rng(11)
    for qs in (1e3, 1e-6):
        assert _attend(q, rng, [400, 90], [2, 1], 16, 16, 1, 4, 64, "e4m3", "bf16", qscale=qs) == 0


def test_reads_what_kv_cache_write_wrote():
    """A cache with one scale per token and head is a block cache with blocks of one token."""
    q = need_gpu()
    rng = np.random.default_rng(12)
    for fmt in ("int8", "e4m3"):
        pages, page, H, D, n = 4, 16, 2, 64, 50
        caches = []
        rows = [torch.from_numpy(rng.normal(size=(n, H, D))).to(torch.bfloat16).cuda() for _ in range(2)]
        for x in rows:
            codes = torch.zeros((pages, page, H, D), dtype=torch.uint8, device="cuda")
            scales = torch.zeros((pages, page, H, 1), device="cuda")
            h = q.make_kv_cache(codes, scales, None, D, fmt, -1)
            q.kv_cache_write(x, None, torch.arange(n, device="cuda"), h, None)
            back = torch.empty((n, H, D), device="cuda")
            q.kv_cache_read(h, None, torch.arange(n, device="cuda"), back, None)
            caches.append((q.make_kv_blocks(codes, scales[..., 0], fmt), host(back.double())))
        x = torch.from_numpy(rng.normal(size=(1, 4, D))).to(torch.bfloat16)
        out = torch.empty((1, 4, D), dtype=torch.bfloat16, device="cuda")
        say("attend to a token cache", fmt)
        q.kv_block_attention(x.cuda(), caches[0][0], caches[1][0], ints([[0, 1, 2, 3]]), ints([n]), ints([0, 1]), out)
        for h in range(4):
            s = caches[0][1][:, h // 2] @ x[0, h].double().numpy() / 8
            w = np.exp(s - s.max())
            w /= w.sum()
            v = caches[1][1][:, h // 2]
            want, mag = w @ v, w @ np.abs(v)
            assert np.all(np.abs(host(out.double())[0, h] - want) <= 2.0 ** -8 * np.abs(want) + 1.01 * (2.0 ** -8 + 2.0 ** -13) * mag)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: its last pages are written and attended to."""
    q = need_gpu()
    pages, page, H, D = 40000, 64, 16, 128
    codes = [torch.zeros((pages, page, H, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((pages, 1, H), device="cuda") for _ in range(2)]
    kb, vb = (q.make_kv_blocks(c, s, "e4m3") for c, s in zip(codes, scales))
    rng = np.random.default_rng(13)
    n = 100
    table = [[pages - 1, pages - 3]]
    k, v = (torch.from_numpy(rng.normal(size=(n, H, D))).float() for _ in range(2))
    say("block cache past 32 bits")
    q.kv_block_write(k.cuda(), v.cuda(), kb, vb, ints(table), ints([n]), ints([0, n]))
    x = torch.from_numpy(rng.normal(size=(1, H, D))).float()
    out = torch.empty((1, H, D), device="cuda")
    q.kv_block_attention(x.cuda(), kb, vb, ints(table), ints([n]), ints([0, 1]), out)
    at = [np.concatenate([host(t[p]) for p in table[0]]) for t in codes]
    sc = [np.repeat(np.concatenate([host(t[p]) for p in table[0]]), page, 0)[:n].astype(float) for t in scales]
    kd, vd = (lowp.e4m3_decode(a[:n]) * s[..., None] for a, s in zip(at, sc))
    for d, x0 in ((kd, k), (vd, v)):
        a = np.abs(x0.double().numpy())
        assert np.all(np.abs(d - x0.double().numpy()) <= 2.0 ** -4 * a + a.max() / 448 * 2.0 ** -9)
    for h in range(H):
        s = kd[:, h] @ x[0, h].double().numpy() * D ** -0.5
        w = np.exp(s - s.max())
        w /= w.sum()
        want, mag = w @ vd[:, h], w @ np.abs(vd[:, h])
        assert np.all(np.abs(host(out.double())[0, h] - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -13 * mag)
    assert sum(int(torch.count_nonzero(s)) for s in scales) == 4 * H


def test_captured_and_replayed():
    """A decode step and a chunk as one graph, replayed with other inputs and lengths; two graphs share
    no workspace of the caller's here."""
    q = need_gpu()
    rng = np.random.default_rng(14)
    H, G, D, page, S = 2, 4, 64, 16, 3
    width = 40
    table = ints(np.arange(S * width).reshape(S, width))
    kb, vb = (BlockCache(q, rng, S * width, page, page, H, D, "int8") for _ in range(2))
    lens, st = ints([1] * S), ints([0, 1, 2, 3])
    kv = torch.zeros((S, 2 * H, D), dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((S, H * G, D), dtype=torch.bfloat16, device="cuda")
    out, want = torch.empty_like(x), torch.empty_like(x)

    def step(o):
        q.kv_block_write(kv[:, :H], kv[:, H:], kb.h, vb.h, table, lens, st)
        q.kv_block_attention(x, kb.h, vb.h, table, lens, st, o)

    step(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(out)
    for turn, n in enumerate(([1, 1, 1], [600, 17, 16], [640, 1, 33], [5, 640, 639])):
        kv.copy_(torch.randn(kv.shape))
        x.copy_(torch.randn(x.shape))
        lens.copy_(ints(n))
        keep = [t.clone() for c in (kb, vb) for t in (c.codes, c.scales)]
        g.replay()
        torch.cuda.synchronize()
        after = [t.clone() for c in (kb, vb) for t in (c.codes, c.scales)]
        for t, k in zip([t for c in (kb, vb) for t in (c.codes, c.scales)], keep):
            t.copy_(k)
        step(want)
        torch.cuda.synchronize()
        assert torch.equal(out, want), turn
        for a, t in zip(after, [t for c in (kb, vb) for t in (c.codes, c.scales)]):
            assert torch.equal(a, t), turn


def test_the_binding_refuses():
    q = need_gpu()
    rng = np.random.default_rng(15)
    kb, vb, other = (BlockCache(q, rng, 2, 16, b, 2, 32, "e4m3") for b in (16, 16, 8))
    x = torch.zeros((3, 2, 32), device="cuda")
    t, n, s = ints([[0], [1]]), ints([3, 3]), ints([0, 1, 3])
    o = torch.empty_like(x)
    for bad in (lambda: q.kv_block_write(x, None, kb.h, None, t.long()[0], n, s),
                lambda: q.kv_block_write(x, None, kb.h, None, t, n[:1], s),
                lambda: q.kv_block_write(x, None, kb.h, None, t, n, s[:2]),
                lambda: q.kv_block_write(x, x, kb.h, other.h, t, n, s),
                lambda: q.kv_block_write(x, x, kb.h, None, t, n, s),
                lambda: q.kv_block_write(x[:, :1], None, kb.h, None, t, n, s),
                lambda: q.kv_block_write(None, None, kb.h, None, t, n, s),
                lambda: q.kv_block_attention(x, kb.h, other.h, t, n, s, o),
                lambda: q.kv_block_attention(x, kb.h, None, t, n, s, o),
                lambda: q.kv_block_attention(x[:, :1], kb.h, vb.h, t, n, s, o[:, :1]),
                lambda: q.kv_block_attention(x, kb.h, vb.h, t, n, s, o[:2]),
                lambda: q.kv_block_attention(x, kb.h, vb.h, t, n, s, o.cpu()),
                lambda: q.kv_block_attention(x, kb.h, vb.h, t.cpu(), n, s, o),
                lambda: q.make_kv_blocks(kb.codes, kb.scales[:, :, :1], "e4m3"),
                lambda: q.make_kv_blocks(kb.codes, kb.scales.repeat(1, 3, 1), "e4m3"),
                lambda: q.make_kv_blocks(kb.codes, kb.scales, "int4")):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q.kv_block_write(x.half(), None, kb.h, None, t, n, s),
                lambda: q.kv_block_write(x, None, kb.h, None, t.long(), n, s),
                lambda: q.kv_block_attention(x, kb.h, vb.h, t, n.long(), s, o),
                lambda: q.kv_block_attention(x, kb.h, vb.h, t, n, s, o.bfloat16())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: q.kv_block_attention(x, kb.h, vb.h, t, n, s, x),
                lambda: q.kv_block_attention(x, kb.h, vb.h, t, n, s, o, window=-1),
                lambda: q.kv_block_attention(x, kb.h, vb.h, t, n, s, o, window=4, causal=False),
                lambda: q.kv_block_write(x, x, kb.h, kb.h, t, n, s)):
        with pytest.raises(q.GPTQError):
            bad()
