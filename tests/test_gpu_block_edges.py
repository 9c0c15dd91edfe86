"""GPU: the cache with a scale per block, its pages and the verification of drafts at the ends of their
ranges, beside each other on streams and in graphs, and together as a serving loop runs them.  Bounds are
those of the operators' own tests."""
import numpy as np
import pytest

from oracle import blocks

from block_util import DT, BlockCache, ints, scattered, starts_of
from gpu_util import host, need_gpu, say, torch
from test_gpu_kv_blocks import _attend, _same_cache
from test_gpu_kv_pages import _pool, _resize
from test_gpu_verify import _case

pytestmark = pytest.mark.gpu

FAR = 2 ** 31 - 1


# ---- many rows of queries

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dim,dt", [(16, "bf16"), (64, "f32"), (96, "bf16"), (128, "f32"), (128, "bf16"), (256, "bf16"), (208, "f32")])
@pytest.mark.parametrize("lens,news,page,block,heads,group,kw", [
    ([70], [37], 16, 16, 1, 1, {}),
    ([1500], [50], 24, 8, 1, 1, {}),                                   # split over keys
    ([1200, 300, 90], [20, 40, 30], 16, 4, 1, 4, {"window": 100, "pad": 3}),
    ([333, 129], [200, 129], 128, 64, 2, 1, {"order": "hpd"}),
    ([260, 5], [3, 300], 1, 1, 1, 1, {"window": 7}),                   # most rows in front of position 0
    ([700, 0], [64, 66], 64, 32, 1, 3, {"causal": False}),
])
def test_tiles_of_rows(fmt, dim, dt, lens, news, page, block, heads, group, kw):
    q = need_gpu()
    rng = np.random.default_rng(sum(lens) + dim)
    assert _attend(q, rng, lens, news, page, block, heads, group, dim, fmt, dt, **kw) == 0


# ---- many sequences

@pytest.mark.parametrize("seqs", [65, 5000])
@pytest.mark.parametrize("most", [1, 6])
def test_many_sequences(seqs, most):
    q = need_gpu()
    rng = np.random.default_rng(seqs + most)
    lens = [int(v) for v in rng.integers(0, 9, size=seqs)]
    news = [int(rng.integers(0, min(n, most) + 1)) for n in lens]
    heads, dim, page, block = 2, 16, 4, 2
    assert _attend(q, rng, lens, news, page, block, heads, 2, dim, "e4m3", "bf16", pad=3) == 0
    table, pages = scattered(rng, lens, page)
    c = BlockCache(q, rng, pages, page, block, heads, dim, "int8")
    want = c.host()
    x = torch.from_numpy(rng.normal(size=(sum(news), heads, dim))).float()
    blocks.write(*want, "int8", x.double().numpy(), table, lens, starts_of(news))
    q.kv_block_write(None, x.cuda(), None, c.h, ints(table), ints(lens), ints(starts_of(news)))
    _same_cache(c, want)


# ---- a call for some of a batch's sequences

@pytest.mark.parametrize("rows", [1, 3, 70])
@pytest.mark.parametrize("dt,fmt", [("bf16", "e4m3"), ("f32", "int8")])
def test_starts_that_begin_later(rows, dt, fmt):
    """starts, lengths and table of the last sequences of a batch, with the whole batch's rows: the others'
    rows, codes and scales stay as they are."""
    q = need_gpu()
    rng = np.random.default_rng(rows)
    lens = [int(v) for v in rng.integers(rows, rows + 200, size=9)]
    news = [rows] * 9
    H, G, D, page, block, skip = 2, 3, 64, 16, 8, 6
    table, pages = scattered(rng, lens, page)
    kb, vb = (BlockCache(q, rng, pages, page, block, H, D, fmt) for _ in range(2))
    st = starts_of(news)
    T = st[-1]
    kv = torch.from_numpy(rng.normal(size=(T, 2 * H, D)) * 4).to(DT[dt])
    x = torch.from_numpy(rng.normal(size=(T, H * G, D))).to(DT[dt])
    want = [c.host() for c in (kb, vb)]
    for w, r in zip(want, (kv[:, :H], kv[:, H:])):
        blocks.write(*w, fmt, r.double().numpy(), table[skip:], lens[skip:], st[skip:])
    some = (ints(table)[skip:], ints(lens)[skip:], ints(st)[skip:])
    d = kv.cuda()
    say("starts that begin later", rows, dt, fmt)
    q.kv_block_write(d[:, :H], d[:, H:], kb.h, vb.h, *some)
    _same_cache(kb, want[0])
    _same_cache(vb, want[1])
    out = torch.full((T, H * G, D), 7.0, dtype=DT[dt], device="cuda")
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    q.kv_block_attention(x.cuda(), kb.h, vb.h, *some, out, info=info)
    assert int(info) == 0
    assert bool((out[:st[skip]] == 7).all())
    ref, _, mag, smax = blocks.attention(x.double().numpy(), *kb.host(), *vb.host(), fmt, table[skip:], lens[skip:], st[skip:])
    got, ref, mag, smax = (v[st[skip]:] for v in (host(out.double()), ref, mag, smax))
    e = 2 * ((D + 8) * 2.0 ** -23 * smax + 2.0 ** -21) + (max(lens) + 16) * 2.0 ** -23
    w, half = (2.0 ** -8, 2.0 ** -8) if dt == "bf16" else (2.0 ** -22, 2.0 ** -24)
    assert np.all(np.abs(got - ref) <= half * np.abs(ref) + (1 + half) * (w * (1 + e) + e)[..., None] * mag + max(lens) * 2.0 ** -122)


def test_verification_of_some_sequences():
    q = need_gpu()
    rng = np.random.default_rng(72)
    counts = [3, 4, 2, 5]
    t, d, ids, u, un = _case(rng, counts, 300)
    st = starts_of(counts)
    a, b, i, uu, nn = t.float().cuda(), d.float().cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(u).cuda(), torch.from_numpy(un).cuda()
    whole = ints([7] * 4), torch.full((st[-1],), 7, dtype=torch.int64, device="cuda")
    some = ints([7] * 2), torch.full((st[-1],), 7, dtype=torch.int64, device="cuda")
    say("verification of some sequences")
    q.verify_drafts(a, b, i, ints(st), uu, nn, *whole)
    q.verify_drafts(a, b, i, ints(st)[2:], uu, nn[2:], *some)
    assert torch.equal(some[0], whole[0][2:]) and torch.equal(some[1][st[2]:], whole[1][st[2]:])
    assert bool((some[1][:st[2]] == 7).all())


# ---- growing blocks, by units of each size

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("heads,dim,block,news", [
    (5, 128, 16, [1, 3]), (9, 48, 32, [40] + [1] * 9), (1, 16, 64, [2, 1]), (6, 64, 128, [1] * 800),                  # 16 lanes
    (5, 128, 64, [1] * 7), (3, 256, 32, [2, 2, 1]), (9, 48, 128, [1, 0, 90, 1]), (5, 128, 64, [9, 4, 3]), (2, 80, 16, [30, 16, 1]),  # a wave
    (3, 128, 128, [40, 20, 70]), (1, 256, 64, [100, 9]),                                                              # four
])
def test_blocks_that_grow(fmt, heads, dim, block, news):
    """Rows 2^-3 .. 2^8 times as large as those in the block, per sequence and head."""
    q = need_gpu()
    rng = np.random.default_rng(heads + dim)
    lens = [n + int(rng.integers(0, 2 * block)) for n in news]
    table, pages = scattered(rng, lens, block)
    kb, vb = (BlockCache(q, rng, pages, block, block, heads, dim, fmt) for _ in range(2))
    want = [c.host() for c in (kb, vb)]
    st = starts_of(news)
    x = rng.normal(size=(sum(news), 2 * heads, dim)) * 2.0 ** rng.integers(-3, 9, size=(sum(news), 2 * heads, 1))
    x = torch.from_numpy(x).to(torch.bfloat16)
    for w, r in zip(want, (x[:, :heads], x[:, heads:])):
        blocks.write(*w, fmt, r.double().numpy(), table, lens, st)
    d = x.cuda()
    say("blocks that grow", fmt, heads, dim, block, news)
    q.kv_block_write(d[:, :heads], d[:, heads:], kb.h, vb.h, ints(table), ints(lens), ints(st))
    _same_cache(kb, want[0])
    _same_cache(vb, want[1])


# ---- lengths and windows at the end of 32 bits

@pytest.mark.parametrize("rows", [1, 80])
@pytest.mark.parametrize("length", [97, 2 ** 30, FAR])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_lengths_past_the_table(rows, length, dt):
    """Keys behind the table's end are not there, and reported; the others are."""
    q = need_gpu()
    rng = np.random.default_rng(41)
    kb, vb = (BlockCache(q, rng, 6, 16, 16, 1, 32, "e4m3") for _ in range(2))
    table, st = ints([[5, 4, 3, 2, 1, 0]]), ints([0, rows])
    x = torch.from_numpy(rng.normal(size=(rows, 2, 32))).to(DT[dt]).cuda()
    out, want = torch.empty_like(x), torch.empty_like(x)
    lse, wlse = (torch.empty((rows, 2), device="cuda") for _ in range(2))
    q.kv_block_attention(x, kb.h, vb.h, table, ints([96]), st, want, lse=wlse, causal=False)
    for causal in (False, True):
        info = torch.zeros(1, dtype=torch.int32, device="cuda")
        say("attend past the table", rows, length, dt, causal)
        q.kv_block_attention(x, kb.h, vb.h, table, ints([length]), st, out, lse=lse, causal=causal, info=info)
        assert int(info) == 1
        last = slice(rows - 1, rows) if causal and length == 97 else slice(0, rows)  # (the rows that see every key)
        assert torch.equal(out[last], want[last]) and torch.equal(lse[last], wlse[last])


def test_writes_past_the_table():
    q = need_gpu()
    rng = np.random.default_rng(42)
    for page, block in ((16, 16), (16, 1), (2 ** 20, 2 ** 20)):
        c = BlockCache(q, rng, 2, page, block, 1, 16, "e4m3") if page == 16 else None
        if c is None:
            codes, scales = torch.zeros((2, page, 1, 16), dtype=torch.uint8, device="cuda"), torch.zeros((2, 1, 1), device="cuda")
            h = q.make_kv_blocks(codes, scales, "e4m3")
        else:
            codes, scales, h = c.codes, c.scales, c.h
        before = codes.clone(), scales.clone()
        x = torch.ones((3, 1, 16), device="cuda")
        info = torch.zeros(1, dtype=torch.int32, device="cuda")
        say("write past the table", page, block)
        q.kv_block_write(x, None, h, None, ints([[0, 1], [1, 0]]), ints([FAR, 2 * page + 1]), ints([0, 2, 3]), info=info)
        assert int(info) == 1
        assert torch.equal(codes, before[0]) and torch.equal(scales, before[1])


@pytest.mark.parametrize("news", [9, 200])
def test_the_widest_window(news):
    """A window of 2^31 - 1 is none, also for a tile whose first rows lie in front of position 0."""
    q = need_gpu()
    rng = np.random.default_rng(43)
    kb, vb = (BlockCache(q, rng, 4, 16, 16, 1, 64, "int8") for _ in range(2))
    x = torch.from_numpy(rng.normal(size=(news, 2, 64))).to(torch.bfloat16).cuda()
    args = (x, kb.h, vb.h, ints([[3, 1, 0, 2]]), ints([5]), ints([0, news]))
    out, want = torch.empty_like(x), torch.empty_like(x)
    say("widest window", news)
    q.kv_block_attention(*args, want)
    q.kv_block_attention(*args, out, window=FAR)
    assert torch.equal(out, want)
    assert bool((want[news - 5:] != 0).any(2).all()) and bool((want[:news - 5] == 0).all())


# ---- pages

def test_growth_beyond_a_small_pool():
    """Thousands more pages are asked for than a pool of a few thousand has: nobody grows."""
    q = need_gpu()
    rows, width, pages = 100, 200, 5000
    table, lens, refs = np.full((rows, width), -1).tolist(), [0] * rows, [0] * pages
    say("growth beyond a small pool")
    got = _resize(q, table, lens, refs, [width] * rows, 1)
    assert got == (table, lens, refs, [-1] * rows, [-1] * rows, 2)
    got = _resize(q, table, lens, refs, [50] * rows, 1)  # all of them
    assert got == blocks.resize(table, lens, refs, [50] * rows, 1) and got[5] == 0


@pytest.mark.parametrize("rows,width,page,pages", [(3, 6000, 1, 20000), (5000, 3, 4, 12000), (1025, 40, 2, 50000)])
def test_large_growth(rows, width, page, pages):
    """More fresh pages than one step holds; rows that share pages across thousands of rows."""
    q = need_gpu()
    rng = np.random.default_rng(rows)
    table, lens, refs = _pool(rng, rows, width, page, 0)
    lens = [n // 3 for n in lens]
    for i, n in enumerate(lens):
        for j in range(blocks.pages_of(n, page), width):
            if table[i][j] >= 0:
                refs[table[i][j]] = 0
                table[i][j] = -1
    refs += [0] * (pages - len(refs))
    for i in range(1, rows, 2):  # pairs of rows half the table apart
        k = (i + rows // 2) % rows
        if k % 2 == 0 and lens[k] > 0:
            for p in table[i]:
                if p >= 0:
                    refs[p] -= 1
            table[i], lens[i] = list(table[k]), lens[k]
            for p in table[i]:
                if p >= 0:
                    refs[p] += 1
    new = [int(rng.integers(n, width * page + 1)) if rng.integers(0, 3) else n + (n < width * page) for n in lens]
    say("large growth", rows, width, page, pages)
    got = _resize(q, table, lens, refs, new, page)
    assert got == blocks.resize(table, lens, refs, new, page)
    assert got[5] == 0


@pytest.mark.parametrize("rows,width,pages", [(900, 9, 8192), (911, 9, 8193), (1024, 8, 8190), (1025, 7, 8000), (20, 400, 7001), (64, 512, 14000), (65, 512, 14000)])
def test_shrinking_and_growing_at_once(rows, width, pages):
    """Pages that some rows give back go to others in the same call (tables that one workgroup settles and
    larger ones; counts of holders that begin off any border)."""
    q = need_gpu()
    rng = np.random.default_rng(rows)
    lens = [int(v) for v in rng.integers(0, width + 1, size=rows)]
    while sum(lens) > pages:
        lens[int(rng.integers(0, rows))] = 0
    order, table, refs, at = rng.permutation(pages), [], [0] * pages, 0
    for n in lens:
        table.append([int(p) for p in order[at:at + n]] + [-1] * (width - n))
        at += n
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] = 1
    # beams of one page's holders among them
    for i in range(0, rows - 1, 5):
        for p in table[i + 1]:
            if p >= 0:
                refs[p] -= 1
        table[i + 1], lens[i + 1] = list(table[i]), lens[i]
        for p in table[i]:
            if p >= 0:
                refs[p] += 1
    page = 3
    lens = [max(page * n - int(rng.integers(0, 3)), 0) if n else 0 for n in lens]
    for turn in range(3):
        new = [int(rng.integers(0, n + 1)) if rng.integers(0, 2) else min(n + int(rng.integers(0, 8)), page * width) for n in lens]
        want = blocks.resize(table, lens, refs, new, page)
        t, n, r = ints(table), ints(lens), ints([0] + refs)[1:]
        src, dst, info = ints([7] * rows), ints([7] * rows), ints([0])
        say("shrink and grow", rows, width, pages, turn)
        q.kv_pages_resize(t, n, r, ints(new), page, src, dst, info=info)
        assert tuple(host(x).tolist() for x in (t, n, r, src, dst)) + (int(info),) == want
        table, lens, refs = want[:3]


# ---- calls beside each other

def _work_of(q, rng, S, rows, ctx):
    """A step of S sequences on caches of its own: (run(outputs), outputs)."""
    H, G, D, page, V = 2, 4, 64, 16, 5000
    width = ctx // page + 1
    table = ints(rng.permutation(S * width).reshape(S, width))
    kb, vb = (BlockCache(q, rng, S * width, page, page, H, D, "e4m3") for _ in range(2))
    lens, st = ints(rng.integers(rows, ctx, size=S)), ints(starts_of([rows] * S))
    kv = torch.from_numpy(rng.normal(size=(S * rows, 2 * H, D))).to(torch.bfloat16).cuda()
    x = torch.from_numpy(rng.normal(size=(S * rows, H * G, D))).to(torch.bfloat16).cuda()
    t, d, ids, u, un = _case(rng, [rows] * S, V)
    t, d, ids, u, un = t.float().cuda(), d.bfloat16().cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(u).cuda(), torch.from_numpy(un).cuda()

    def outputs():
        return [torch.zeros_like(x), ints([0] * S), torch.zeros_like(ids), torch.zeros(len(ids), device="cuda")]

    def run(o):
        q.kv_block_write(kv[:, :H], kv[:, H:], kb.h, vb.h, table, lens, st)
        q.kv_block_attention(x, kb.h, vb.h, table, lens, st, o[0])
        q.verify_drafts(t, d, ids, st, u, un, o[1], o[2], logprobs=o[3])

    return run, outputs, (kb.codes, kb.scales, vb.codes, vb.scales)


def test_two_streams_at_once():
    """Splits and their joins on streams that are not the default one, beside each other."""
    q = need_gpu()
    rng = np.random.default_rng(51)
    work = [_work_of(q, rng, 2, 4, 9000), _work_of(q, rng, 3, 30, 6000)]
    want = []
    for run, outputs, _ in work:
        o = outputs()
        run(o)  # (a second write of the same rows changes nothing more)
        run(o)
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = [w[1]() for w in work]
    torch.cuda.synchronize()
    say("two streams at once")
    for _ in range(4):
        for s, (run, _, _), o in zip(streams, work, got):
            with torch.cuda.stream(s):
                run(o)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_two_graphs_with_one_workspace():
    """Two captured calls that a caller gives the same workspace, replayed in turn."""
    q = need_gpu()
    rng = np.random.default_rng(52)
    H, G, D, page, width = 2, 4, 128, 16, 300
    kb, vb = (BlockCache(q, rng, 2 * width, page, page, H, D, "int8") for _ in range(2))
    table = ints(np.arange(2 * width).reshape(2, width))
    cases = []
    for rows in (1, 40):  # both kernels
        x = torch.from_numpy(rng.normal(size=(2 * rows, H * G, D))).to(torch.bfloat16).cuda()
        cases.append((x, ints([4000, 4800]), ints([0, rows, 2 * rows])))
    need = max(q.kv_block_attention_workspace_size(kb.h, H * G, torch.bfloat16, len(x), 2, width) for x, _, _ in cases)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs, wants, graphs = [], [], []
    for x, n, s in cases:
        out, want = torch.zeros_like(x), torch.zeros_like(x)
        q.kv_block_attention(x, kb.h, vb.h, table, n, s, want, ws=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.kv_block_attention(x, kb.h, vb.h, table, n, s, out, ws=ws)
        outs.append(out), wants.append(want), graphs.append(g)
    say("two graphs with one workspace")
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, wants):
            assert torch.equal(o, w)
            o.zero_()


# ---- together

def test_a_serving_loop():
    """Two prompts, forked to beams; then steps of three drafts each: pages for them, copies of shared
    pages, writes, attention, verification, and the refused drafts' pages back.  Every state equals the
    oracle's; the step as a graph gives what its eager calls gave."""
    q = need_gpu()
    rng = np.random.default_rng(61)
    H, G, D, page, block, width, V, d = 2, 2, 32, 8, 4, 12, 200, 3
    prompts, beams = [21, 10], [0, 0, 0, 1, 1]
    S, B = len(prompts), len(beams)
    pages = 60
    caches = [BlockCache(q, rng, pages, page, block, H, D, f) for f in ("e4m3", "e4m3")]
    other = torch.zeros((pages, page, H, D), dtype=torch.uint8, device="cuda"), torch.ones((pages, page, H, 1), device="cuda")
    layer = q.make_kv_cache(*other, None, D, "int8", -1)  # another layer's cache, with a scale a token
    want = [c.host() for c in caches]
    kb, vb = (c.h for c in caches)
    t, n, r = ints(np.full((S, width), -1)), ints([0] * S), ints([0] * pages)
    src, dst = ints([0] * S), ints([0] * S)
    say("serving loop: prompts")
    q.kv_pages_resize(t, n, r, ints(prompts), page, src, dst)
    table, lens, refs = blocks.resize(np.full((S, width), -1).tolist(), [0] * S, [0] * pages, prompts, page)[:3]
    T = sum(prompts)
    kv = torch.from_numpy(rng.normal(size=(T, 2 * H, D))).to(torch.bfloat16)
    q.kv_block_write(kv[:, :H].cuda(), kv[:, H:].cuda(), kb, vb, t, n, ints(starts_of(prompts)))
    for w, x in zip(want, (kv[:, :H], kv[:, H:])):
        blocks.write(*w, "e4m3", x.double().numpy(), table, lens, starts_of(prompts))
    t2, n2, r2 = ints(np.full((B, width), 7)), ints([7] * B), ints([7] * pages)
    q.kv_pages_fork(t, n, r, ints(beams), page, t2, n2, r2)
    table, lens, refs = blocks.fork(table, lens, refs, beams, page)

    T = B * (d + 1)
    st, info = starts_of([d + 1] * B), torch.zeros(1, dtype=torch.int32, device="cuda")
    starts, src, dst, acc = ints(st), ints([0] * B), ints([0] * B), ints([0] * B)
    kv = torch.zeros((T, 2 * H, D), dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((T, H * G, D), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(x)
    target, draft = (torch.zeros((T, V), device="cuda") for _ in range(2))
    ids, toks = (torch.zeros(T, dtype=torch.int64, device="cuda") for _ in range(2))
    u, un = torch.zeros(T, device="cuda"), torch.zeros(B, device="cuda")
    state = [t2, n2, r2, caches[0].codes, caches[0].scales, caches[1].codes, caches[1].scales, *other]

    def step():
        q.kv_pages_resize(t2, n2, r2, n2 + (d + 1), page, src, dst, info=info)
        q.kv_pages_copy([kb, vb, layer], src, dst, info=info)
        q.kv_block_write(kv[:, :H], kv[:, H:], kb, vb, t2, n2, starts, info=info)
        q.kv_block_attention(x, kb, vb, t2, n2, starts, out, info=info)
        q.verify_drafts(target, draft, ids, starts, u, un, acc, toks)
        q.kv_pages_resize(t2, n2, r2, n2 - (d - acc), page, src, dst, info=info)

    graph = None
    for turn in range(5):
        a, b, i, uu, nn = _case(rng, [d + 1] * B, V)
        a, b = a.float(), b.float()
        rows = torch.from_numpy(rng.normal(size=(T, 2 * H, D))).to(torch.bfloat16)
        xs = torch.from_numpy(rng.normal(size=(T, H * G, D))).to(torch.bfloat16)
        for to, v in ((target, a), (draft, b), (ids, torch.from_numpy(i)), (u, torch.from_numpy(uu)), (un, torch.from_numpy(nn)), (kv, rows), (x, xs)):
            to.copy_(v)
        keep = [v.clone() for v in state]
        say("serving loop: step", turn)
        step()
        torch.cuda.synchronize()
        after = [v.clone() for v in state] + [out.clone(), acc.clone(), toks.clone()]
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        for v, k in zip(state, keep):
            v.copy_(k)
        graph.replay()
        torch.cuda.synchronize()
        for v, w in zip(state + [out, acc, toks], after):
            assert torch.equal(v, w), turn
        assert int(info) == 0
        # the oracle's step
        table, lens, refs, ws, wd, _ = blocks.resize(table, lens, refs, [v + d + 1 for v in lens], page)
        for s, to in zip(ws, wd):
            if s >= 0:
                for w in want:
                    w[0][to], w[1][to] = w[0][s], w[1][s]
        for w, v in zip(want, (rows[:, :H], rows[:, H:])):
            blocks.write(*w, "e4m3", v.double().numpy(), table, lens, st)
        ref, _, mag, _ = blocks.attention(xs.double().numpy(), *want[0], *want[1], "e4m3", table, lens, st)
        assert np.all(np.abs(host(out.double()) - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * (2.0 ** -8 + 2.0 ** -13) * mag)
        wacc, wtok, _, margin = blocks.verify(a.double().numpy(), b.double().numpy(), i, st, uu.astype(float), nn.astype(float))
        assert margin > 1e-9
        assert np.array_equal(host(acc), wacc) and np.array_equal(host(toks), wtok)
        table, lens, refs = blocks.resize(table, lens, refs, [v - (d - int(k)) for v, k in zip(lens, wacc)], page)[:3]
        assert (host(t2).tolist(), host(n2).tolist(), host(r2).tolist()) == (table, lens, refs)
        for c, w in zip(caches, want):
            _same_cache(c, w)


# ---- NaN among many rows

@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("page,block", [(64, 64), (10, 5)])
@pytest.mark.parametrize("dt,dim,news", [("bf16", 128, 100), ("bf16", 64, 300), ("f32", 128, 40), ("bf16", 256, 50)])
def test_nan_in_tiles(dt, dim, news, page, block, window):
    """A NaN among the values reaches the rows that see it, in tiles that all rows see as in the others."""
    q = need_gpu()
    rng = np.random.default_rng(71)
    n = 330
    table, pages = scattered(rng, [n], page)
    kb, vb = (BlockCache(q, rng, pages, page, block, 1, dim, "e4m3") for _ in range(2))
    x = torch.from_numpy(rng.normal(size=(news, 2, dim))).to(DT[dt]).cuda()
    args = (ints(table), ints([n]), ints([0, news]))
    clean, out = torch.empty_like(x), torch.empty_like(x)
    q.kv_block_attention(x, kb.h, vb.h, *args, clean, window=window)
    for p, col in ((3, 5), (n - news + 20, dim - 1), (n - 1, 0)):
        place = table[0][p // page], p % page, 0, col
        kept = vb.codes[place].clone()
        vb.codes[place] = 0x7F
        say("nan in tiles", dt, dim, news, page, window, p)
        q.kv_block_attention(x, kb.h, vb.h, *args, out, window=window)
        vb.codes[place] = kept
        pos = torch.arange(n - news, n, device="cuda")
        want = torch.zeros(x.shape, dtype=torch.bool, device="cuda")
        want[(pos >= p) & ((pos < p + window) if window else (pos >= 0)), :, col] = True
        assert torch.equal(torch.isnan(out), want), p
        assert torch.equal(out[~want], clean[~want]), p


# ---- rows off any border

@pytest.mark.parametrize("rows", [2, 60])
@pytest.mark.parametrize("dt,fmt", [("bf16", "e4m3"), ("bf16", "int8"), ("f32", "e4m3")])
@pytest.mark.parametrize("dim", [16, 112, 128, 256])
def test_unaligned_rows(rows, dt, fmt, dim):
    """Rows, queries and outputs of matrices with odd strides, beginning off 16-byte borders: bit for bit what
    aligned ones give; nothing beside them changes."""
    q = need_gpu()
    rng = np.random.default_rng(rows + dim)
    lens, H, G, page = [rows + 37, rows + 5], 2, 2, 16
    table, pages = scattered(rng, lens, page)
    caches = [[BlockCache(q, np.random.default_rng(s), pages, page, page, H, dim, fmt) for s in (1, 2)] for _ in range(2)]
    args = (ints(table), ints(lens), ints([0, rows, 2 * rows]))
    kv = torch.from_numpy(rng.normal(size=(2 * rows, 2 * H, dim))).to(DT[dt]).cuda()
    x = torch.from_numpy(rng.normal(size=(2 * rows, H * G, dim))).to(DT[dt]).cuda()

    def odd(t, fill=3.0):
        wide = torch.full((t.shape[0], t.shape[1], dim + 5), fill, dtype=t.dtype, device="cuda")
        wide[..., 3:dim + 3] = t
        return wide, wide[..., 3:dim + 3]

    outs = []
    say("unaligned rows", rows, dt, fmt, dim)
    for (kb, vb), f in zip(caches, (lambda t: (t, t), odd)):
        k, v, y = (f(t.contiguous())[1] for t in (kv[:, :H], kv[:, H:], x))
        wide, out = f(torch.zeros_like(x))
        q.kv_block_write(k, v, kb.h, vb.h, *args)
        q.kv_block_attention(y, kb.h, vb.h, *args, out)
        outs.append(out)
        if wide is not out:
            assert bool((wide[..., :3] == 3).all()) and bool((wide[..., dim + 3:] == 3).all())
    for a, b in zip(*caches):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    assert torch.equal(*outs)
