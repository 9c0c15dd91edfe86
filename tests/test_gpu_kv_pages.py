"""GPU: pages of a cache that are forked, resized, compacted and copied, against the oracle's lists."""
import numpy as np
import pytest

from oracle import blocks

from block_util import BlockCache, ints
from gpu_util import host, need_gpu, say, torch

pytestmark = pytest.mark.gpu


def _pool(rng, rows, width, page, spare, full=False):
    """Rows of random lengths whose pages are scattered over a pool."""
    lens = [width * page if full else int(rng.integers(0, width * page + 1)) for _ in range(rows)]
    need = [blocks.pages_of(n, page) for n in lens]
    pages = max(sum(need) + spare, 1)
    order = rng.permutation(pages)
    table, refs, at = [], [0] * pages, 0
    for n in need:
        own = [int(p) for p in order[at:at + n]]
        at += n
        for p in own:
            refs[p] = 1
        table.append(own + [-1] * (width - n))
    return table, lens, refs


def _fork(q, table, lens, refs, parents, page):
    R, W = len(parents), len(table[0])
    nt, nl, nr = ints(np.full((R, W), 77)), ints([77] * R), ints([77] * len(refs))
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    q.kv_pages_fork(ints(table), ints(lens), ints(refs), ints(parents), page, nt, nl, nr, info=info)
    return host(nt).tolist(), host(nl).tolist(), host(nr).tolist(), int(info)


def _resize(q, table, lens, refs, new, page):
    t, n, r = ints(table), ints(lens), ints(refs)
    src, dst = ints([77] * len(table)), ints([77] * len(table))
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    q.kv_pages_resize(t, n, r, ints(new), page, src, dst, info=info)
    return tuple(host(x).tolist() for x in (t, n, r, src, dst)) + (int(info),)


@pytest.mark.parametrize("rows,width,page,beams", [(1, 1, 1, 1), (5, 4, 16, 3), (40, 70, 7, 8), (300, 9, 64, 4), (1500, 3, 2, 5)])
def test_fork_and_resize(rows, width, page, beams):
    """Forks and growth again and again: every step's tables, holders and copies equal the lists'."""
    q = need_gpu()
    rng = np.random.default_rng(rows + width)
    table, lens, refs = _pool(rng, rows, width, page, rows * width + 10)
    refs[refs.index(0)] = 2  # a page that others hold
    for step in range(5):
        parents = [int(min(rows - 1, max(-1, i - i % beams + rng.integers(-1, beams)))) for i in range(rows)]
        say("fork", rows, width, page, step)
        got = _fork(q, table, lens, refs, parents, page)
        table, lens, refs = blocks.fork(table, lens, refs, parents, page)
        assert got == (table, lens, refs, 0)
        new = []
        for n in lens:
            kind = rng.integers(0, 8)
            new.append(-1 if kind == 0 else 0 if kind == 1 else int(rng.integers(0, width * page + 1)) if kind == 2
                       else n if kind == 3 else min(n + 1, width * page) if kind < 6
                       else min(n + int(rng.integers(1, 3 * page + 2)), width * page))
        if step == 2:
            new[0] = width * page + 1  # more than the row can hold
        say("resize", rows, width, page, step)
        got = _resize(q, table, lens, refs, new, page)
        want = blocks.resize(table, lens, refs, new, page)
        assert got == want
        table, lens, refs = want[:3]
        assert all(n >= 0 for n in refs)


def test_resize_runs_out_of_pages():
    """Shorter rows give their pages back, then nobody grows; with one page more they all do."""
    q = need_gpu()
    table, lens, refs = [[0, 1, -1], [2, -1, -1], [3, 4, -1]], [8, 4, 7], [1] * 5
    new = [4, 9, 9]  # frees page 1; two and one pages are needed
    say("resize out of pages")
    got = _resize(q, table, lens, refs, new, 4)
    assert got == blocks.resize(table, lens, refs, new, 4) and got[5] == 2
    assert got[1] == [4, 4, 7] and got[2][1] == 0
    got = _resize(q, table, lens, refs + [0, 0], new, 4)
    assert got == blocks.resize(table, lens, refs + [0, 0], new, 4) and got[5] == 0
    assert got[0] == [[0, -1, -1], [2, 1, 5], [3, 4, 6]]


def test_the_last_holder_keeps_a_shared_page():
    q = need_gpu()
    table, lens = [[3, 7], [3, 7], [3, 7], [3, 7]], [6, 6, 6, 6]
    refs = [0, 1, 0, 4, 0, 0, 0, 4]
    say("resize shared")
    for new, src in (([7, 7, 7, 7], [7, 7, 7, -1]), ([7, -1, 7, -1], [7, -1, 7, -1]), ([7, 0, 0, 4], [-1] * 4), ([8, 0, 6, 4], [7, -1, -1, -1])):
        got = _resize(q, table, lens, refs, new, 4)
        assert got == blocks.resize(table, lens, refs, new, 4)
        assert got[3] == src, new
    refs[7] = 5  # and somebody outside the table
    got = _resize(q, table, lens, refs, [7] * 4, 4)
    assert got == blocks.resize(table, lens, refs, [7] * 4, 4) and got[3] == [7] * 4


def test_bad_entries_are_left_out():
    q = need_gpu()
    say("fork and resize with bad entries")
    nt, nl, nr, info = _fork(q, [[0, 5], [1, -1]], [8, 4], [1, 1, 0], [1, 9, -3], 4)
    assert info == 1 and nl == [4, 0, 0] and nt == [[1, -1], [-1, -1], [-1, -1]] and nr == [0, 1, 0]
    t, n, r, src, dst, info = _resize(q, [[0, 9], [-1, -1]], [8, 3], [1, 0, 0], [2, 4], 4)
    assert info == 1 and t[0] == [0, -1] and n == [2, 4] and src == [-1, -1]


@pytest.mark.parametrize("rows,width,page,spare", [(1, 1, 1, 0), (3, 5, 4, 40), (64, 30, 16, 5000), (20, 3, 2, 0), (0, 4, 4, 9), (500, 200, 1, 70000)])
def test_compact(rows, width, page, spare):
    q = need_gpu()
    rng = np.random.default_rng(rows + spare)
    table, lens, refs = _pool(rng, rows, width, page, spare, full=spare == 0) if rows else ([], [], [0, 2, 0, 0, 1, 0, 3, 0, 0])
    refs = [int(n * rng.integers(1, 4)) for n in refs]
    N, cap = len(refs), len(refs) // 2 + 3
    nt, nr, src, dst, count = (ints(np.full((rows, width), 77)), ints([77] * N), ints([77] * cap), ints([77] * cap), ints([77]))
    say("compact", rows, width, page, spare)
    q.kv_pages_compact(ints(np.array(table).reshape(rows, width)), ints(refs), nt, nr, src, dst, count)
    wt, wr, ws, wd, L = blocks.compact(table, refs)
    assert int(count) == L
    assert host(nt).tolist() == wt and host(nr).tolist() == wr
    assert host(src).tolist() == ws + [-1] * (cap - len(ws)) and host(dst).tolist() == wd + [-1] * (cap - len(wd))


@pytest.mark.parametrize("order", ["phd", "hpd"])
def test_copy(order):
    """Pairs in every array of several caches of different kinds; negative pairs, a pair onto itself and
    pages that are none are left out; nothing else changes."""
    q = need_gpu()
    rng = np.random.default_rng(21)
    pages = 50
    caches = [BlockCache(q, rng, pages, p, b, h, d, f, order)
              for p, b, h, d, f in ((16, 16, 8, 128, "e4m3"), (20, 5, 3, 80, "int8"), (1, 1, 1, 16, "int8"), (64, 32, 2, 64, "e4m3"))]
    ng = 3
    int4 = [torch.randint(0, 256, (pages, 4, 2, 36), dtype=torch.uint8, device="cuda"),
            torch.randn((pages, 4, 2, ng), device="cuda"), torch.randint(0, 16, (pages, 4, 2, ng), dtype=torch.uint8, device="cuda")]
    handles = [c.h for c in caches] + [q.make_kv_cache(*int4, 72, "int4", 32)] + [c.h for c in caches] * 8  # (more arrays than a launch takes)
    tensors = [t for c in caches for t in (c.codes, c.scales)] + int4
    order_ = rng.permutation(pages)
    src = [int(p) for p in order_[:12]] + [-1, 3, int(order_[40])]
    dst = [int(p) for p in order_[12:24]] + [4, -1, int(order_[40])]
    before = [t.clone() for t in tensors]
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    say("copy pages", order)
    q.kv_pages_copy(handles, ints(src), ints(dst), info=info)
    assert int(info) == 0
    for t, b in zip(tensors, before):
        for s, d in zip(src, dst):
            if s >= 0 and d >= 0:
                b[d] = b[s].clone()
        assert torch.equal(t, b)
    q.kv_pages_copy(handles[:1], ints([pages, 1]), ints([0, pages + 7]), info=info)
    assert int(info) == 1
    assert torch.equal(tensors[0], before[0])
    q.kv_pages_copy([], ints([1]), ints([2]))
    q.kv_pages_copy(handles, ints([]), ints([]))


def test_step_captured_and_replayed():
    """A beam step (fork, growth, copies) as one graph, its inputs changed between the replays."""
    q = need_gpu()
    rng = np.random.default_rng(22)
    R, W, page = 12, 8, 16
    table, lens, refs = _pool(rng, R, W, page, 60)
    lens = [min(n, W * page - 5) for n in lens]
    N = len(refs)
    t, n, r = ints(table), ints(lens), ints(refs)
    t2, n2, r2 = torch.empty_like(t), torch.empty_like(n), torch.empty_like(r)
    par, new, src, dst = (ints([0] * R) for _ in range(4))
    cache = BlockCache(q, rng, N, page, page, 2, 32, "e4m3")

    def step():
        q.kv_pages_fork(t, n, r, par, page, t2, n2, r2)
        q.kv_pages_resize(t2, n2, r2, new, page, src, dst)
        q.kv_pages_copy([cache.h], src, dst)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for turn in range(4):
        table, lens, refs = _pool(rng, R, W, page, N)
        extra = N - len(refs)
        table = [[p % N for p in row] if extra else row for row in table]
        table, lens, refs = _fit(rng, R, W, page, N)
        parents = [int(v) for v in rng.integers(-1, R, size=R)]
        mid = blocks.fork(table, lens, refs, parents, page)
        grow = [min(v + 1, W * page) for v in mid[1]]
        want = blocks.resize(*mid, grow, page)
        t.copy_(ints(table)); n.copy_(ints(lens)); r.copy_(ints(refs)); par.copy_(ints(parents)); new.copy_(ints(grow))
        before = cache.codes.clone()
        g.replay()
        torch.cuda.synchronize()
        assert (host(t2).tolist(), host(n2).tolist(), host(r2).tolist(), host(src).tolist(), host(dst).tolist()) == want[:5], turn
        for s, d in zip(*want[3:5]):
            if s >= 0:
                before[d] = before[s].clone()
        assert torch.equal(cache.codes, before)


def _fit(rng, R, W, page, N):
    """A pool of exactly N pages."""
    while True:
        table, lens, refs = _pool(rng, R, W, page, 0)
        used = sum(n > 0 for n in refs)
        if used + R <= N:
            break
    to = rng.permutation(N)
    out = [0] * N
    for p, k in enumerate(refs):
        out[int(to[p])] = k
    return [[int(to[p]) if p >= 0 else -1 for p in row] for row in table], lens, out


def test_the_binding_refuses():
    q = need_gpu()
    t, n, r = ints([[0, 1], [2, -1]]), ints([8, 4]), ints([1, 1, 1, 0])
    t2, n2, r2 = torch.empty_like(t), torch.empty_like(n), torch.empty_like(r)
    s, d = ints([0, 0]), ints([0, 0])
    for bad in (lambda: q.kv_pages_fork(t, n, r, n, 4, t2[:, :1], n2, r2),
                lambda: q.kv_pages_fork(t, n[:1], r, n, 4, t2, n2, r2),
                lambda: q.kv_pages_fork(t, n, r, n, 4, t2, n2, r2[:2]),
                lambda: q.kv_pages_resize(t, n, r, n2, 4, s[:1], d),
                lambda: q.kv_pages_resize(t.cpu(), n, r, n2, 4, s, d),
                lambda: q.kv_pages_compact(t, r, t2, r2, s[:1], d, n),
                lambda: q.kv_pages_compact(t, r, t2[:1], r2, s, d, n),
                lambda: q.kv_pages_copy([], s, d[:1])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q.kv_pages_fork(t, n, r, n, 4, t, n2, r2),
                lambda: q.kv_pages_fork(t, n, r, n, 4, t2, n2, r),
                lambda: q.kv_pages_fork(t, n, r, n, 0, t2, n2, r2),
                lambda: q.kv_pages_resize(t, n, r, n, 4, s, d),
                lambda: q.kv_pages_resize(t, n, r, n2, 4, s, s),
                lambda: q.kv_pages_compact(t, r, t, r2, s, d, n)):
        with pytest.raises(q.GPTQError):
            bad()
