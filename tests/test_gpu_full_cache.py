"""GPU: the decode step of the README, as it stands there, with pages enough and with too few; and its captured form."""
import pathlib
import re

import numpy as np
import pytest

from block_util import BlockCache, ints, scattered, starts_of
from gpu_util import host, need_gpu, say, torch

pytestmark = pytest.mark.gpu

README = pathlib.Path(__file__).resolve().parents[1] / "README.md"


def _step_of_the_readme():
    blocks = re.findall(r"```python\n(.*?)```", README.read_text(), re.S)
    (step,) = [b for b in blocks if "kv_pages_resize" in b]
    return compile(step, "README.md", "exec")


def _batch(q, spare, seed):
    """Three sequences, the first two of which share their pages, and what a step of 1 + 2 + 3 rows needs."""
    rng = np.random.default_rng(seed)
    page, heads, group, dim, vocab, counts = 16, 2, 3, 64, 50, [1, 2, 3]
    lens = [40, 40, 31]
    table, pages = scattered(rng, lens, page, spare=0, width=8)
    owned = {p for p in table[1] if p >= 0}
    free = sorted(owned)[:spare]  # the second row holds the first one's pages: its own are free, `spare` of them
    refs = [0] * pages
    table[1] = list(table[0])
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] += 1
    for p in owned - set(free):
        refs[p] = 1  # somebody else's
    T = sum(counts)
    keys, values = (BlockCache(q, rng, pages, page, page, heads, dim, "e4m3") for _ in range(2))
    x = lambda *s: torch.from_numpy(rng.normal(size=s)).cuda().bfloat16()  # noqa: E731
    n = dict(q=q, table=ints(table), lengths=ints(lens), refs=ints(refs), rows=ints(counts), page_size=page, src=ints([0] * 3), dst=ints([0] * 3),
             info=ints([0]), caches=[keys.h, values.h], K=x(T, heads, dim), V=x(T, heads, dim), keys=keys.h, values=values.h,
             starts=ints(starts_of(counts)), Q=x(T, heads * group, dim), out=torch.zeros((T, heads * group, dim), dtype=torch.bfloat16, device="cuda"),
             target_logits=x(T, vocab), draft_logits=x(T, vocab), ids=torch.from_numpy(rng.integers(0, vocab, size=T)).cuda(),
             u=torch.from_numpy(rng.random(T)).float().cuda(), u_next=torch.from_numpy(rng.random(3)).float().cuda(), accepted=ints([0] * 3),
             tokens=torch.zeros(T, dtype=torch.int64, device="cuda"), drafts=ints([0, 1, 2]))
    kept = dict(table=n["table"], lengths=n["lengths"], refs=n["refs"], kc=keys.codes, ks=keys.scales, vc=values.codes, vs=values.scales)
    return n, kept


def _copies(kept):
    torch.cuda.synchronize()
    return {k: t.clone() for k, t in kept.items()}


def _same(kept, before):
    torch.cuda.synchronize()
    return [k for k, t in kept.items() if not torch.equal(t, before[k])]


# the rows grow inside of a shared page (one copy: the last holder keeps it) and past a page's end (one more)
NEED = 2


@pytest.mark.parametrize("spare", [0, NEED - 1])
def test_the_readme_step_in_a_full_cache(spare):
    """Pages run out: the step ends, and cache, tables and lengths are as they were."""
    q = need_gpu()
    names, kept = _batch(q, spare, 3)
    before = _copies(kept)
    say("README step, full", spare)
    with pytest.raises(MemoryError):
        exec(_step_of_the_readme(), names)
    assert _same(kept, before) == []


def test_the_readme_step():
    q = need_gpu()
    names, kept = _batch(q, NEED, 4)
    before = _copies(kept)
    say("README step")
    exec(_step_of_the_readme(), names)
    changed = _same(kept, before)
    assert set(changed) == set(kept)
    accepted = host(names["accepted"])
    assert np.array_equal(host(kept["lengths"]), host(before["lengths"]) + 1 + accepted)
    assert int(names["info"]) == 0


def test_the_captured_step_in_a_cache_that_fills():
    """The captured form: a step without pages writes nothing and leaves every length as it is."""
    q = need_gpu()
    names, kept = _batch(q, 3, 5)
    n = type("names", (), names)

    def step():
        n.info.zero_()
        q.kv_pages_resize(n.table, n.lengths, n.refs, n.lengths + n.rows, n.page_size, n.src, n.dst, info=n.info)
        ok = ((n.info & 2) == 0).int()
        starts = n.starts * ok
        q.kv_pages_copy(n.caches, n.src, n.dst)
        q.kv_block_write(n.K, n.V, n.keys, n.values, n.table, n.lengths, starts)
        q.kv_block_attention(n.Q, n.keys, n.values, n.table, n.lengths, starts, n.out)
        q.verify_drafts(n.target_logits, n.draft_logits, n.ids, starts, n.u, n.u_next, n.accepted, n.tokens)
        q.kv_pages_resize(n.table, n.lengths, n.refs, n.lengths - (n.drafts - n.accepted) * ok, n.page_size, n.src, n.dst)

    say("captured step, filling")
    state = _copies(kept)
    step()  # (loads what it needs)
    torch.cuda.synchronize()
    for k, t in kept.items():
        t.copy_(state[k])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    torch.cuda.synchronize()
    assert _same(kept, state) == []
    full = 0
    for turn in range(60):
        before = _copies(kept)
        free = int((before["refs"] == 0).sum())
        g.replay()
        torch.cuda.synchronize()
        changed = _same(kept, before)
        if int(n.info) & 2:
            full += 1
            assert changed == [], turn
            assert np.all(host(n.accepted) == 0)
        else:
            assert full == 0 and "lengths" in changed and "kc" in changed, turn
            assert np.array_equal(host(kept["lengths"]), host(before["lengths"]) + 1 + host(n.accepted)), turn
        assert free >= int((kept["refs"] == 0).sum())
        if full == 4:
            break
    assert full == 4
