"""Pins of the oracle of the block cache, its pages and drafted tokens: closed forms, special cases,
invariants, brute force."""
import numpy as np
import pytest

from oracle import blocks, lowp


@pytest.mark.parametrize("fmt,steps", [("int8", 0.5), ("e4m3", 16.0)])
def test_write_of_whole_blocks(fmt, steps):
    """A block that begins anew: the kv_cache_write grid over the whole block."""
    rng = np.random.default_rng(0)
    x = rng.normal(size=(8, 2, 16)).astype(np.float32).astype(float)
    codes, scales = np.zeros((3, 4, 2, 16), np.uint8), np.zeros((3, 2, 2))
    assert not blocks.write(codes, scales, fmt, x, [[2, 0]], [8], [0, 8])
    for b in range(4):
        for h in range(2):
            part = x[2 * b:2 * b + 2, h]
            c, s, _ = lowp.kv_quantize(part.reshape(1, -1), fmt, -1, False)
            p, o = [2, 2, 0, 0][b], 2 * (b % 2)
            assert np.array_equal(codes[p, o:o + 2, h].reshape(-1), c[0])
            assert scales[p, b % 2, h] == s[0, 0]
            got = blocks.values(codes[p, o:o + 2, h], fmt) * scales[p, b % 2, h]
            assert np.all(np.abs(got - part) <= steps * s[0, 0] * (1 + 2.0 ** -15))
    assert np.all(codes[1] == 0)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_growth(fmt):
    """A row of 10 behind a row of 1: the scale doubles until it covers it, the first row keeps its
    values (e4m3 above its subnormals) or loses half a step."""
    codes, scales = np.zeros((1, 4, 1, 16), np.uint8), np.zeros((1, 1, 1))
    x = np.linspace(0.5, 1.0, 16).reshape(1, 1, 16)
    blocks.write(codes, scales, fmt, x, [[0]], [1], [0, 1])
    before, s0 = blocks.values(codes[0, 0, 0], fmt) * scales[0, 0, 0], scales[0, 0, 0]
    blocks.write(codes, scales, fmt, 10 * x, [[0]], [2], [0, 1])
    assert scales[0, 0, 0] == 16 * s0
    after = blocks.values(codes[0, 0, 0], fmt) * scales[0, 0, 0]
    if fmt == "e4m3":
        assert np.array_equal(after, before)
    else:
        assert np.all(np.abs(after - before) <= 8 * s0)
    blocks.write(codes, scales, fmt, x, [[0]], [3], [0, 1])
    assert scales[0, 0, 0] == 16 * s0  # large enough
    blocks.write(codes, scales, fmt, x, [[0]], [1], [0, 1])
    assert scales[0, 0, 0] == s0  # begun anew


def test_attention_of_equal_and_single_keys():
    rng = np.random.default_rng(1)
    kc, vc = (rng.integers(0, 256, size=(2, 4, 1, 16), dtype=np.uint8) for _ in range(2))
    s = np.full((2, 2, 1), 0.5)
    q = np.zeros((3, 2, 16))
    out, lse, mag, _ = blocks.attention(q, kc, s, vc, s, "int8", [[1, 0]], [6], [0, 3])
    v = (np.concatenate([vc[1, :, 0], vc[0, :, 0]]).astype(float) - 128) * 0.5
    for r in range(3):
        assert np.allclose(out[r, 1], v[:4 + r].mean(0)) and np.isclose(lse[r, 0], np.log(4 + r))
    out, lse, _, _ = blocks.attention(rng.normal(size=(3, 2, 16)), kc, s, vc, s, "int8", [[1, 0]], [6], [0, 3], window=1)
    assert np.allclose(out[:, 0], v[3:6])
    out, lse, _, _ = blocks.attention(q, kc, s, vc, s, "int8", [[1, 0]], [2], [0, 3])
    assert np.all(out[0] == 0) and np.all(np.isneginf(lse[0])) and np.allclose(out[1, 0], v[0])


def test_pages_keep_their_holders():
    """After any forks, growth and compaction: a page's holders are the rows that list it, no two rows
    share a page that either may write, and every listed page is in use."""
    rng = np.random.default_rng(2)
    page, width, R = 4, 6, 9
    table, lens, refs = [[-1] * width for _ in range(R)], [0] * R, [0] * 60
    for step in range(60):
        parents = [int(v) for v in rng.integers(-1, R, size=R)]
        table, lens, refs = blocks.fork(table, lens, refs, parents, page)
        before = [list(r) for r in table]
        new = [int(min(width * page, max(0, n + rng.integers(-3, 7)))) for n in lens]
        old = list(lens)
        table, lens, refs, src, dst, info = blocks.resize(table, lens, refs, new, page)
        assert info in (0, 2)
        for s, d in zip(src, dst):
            assert (s < 0) == (d < 0) and (s < 0 or (refs[s] > 0 and refs[d] == 1))
        held = np.zeros(60, int)
        for r, n in zip(table, lens):
            k = blocks.pages_of(n, page)
            assert all(p >= 0 for p in r[:k]) and all(p == -1 for p in r[k:])
            held += np.bincount(r[:k], minlength=60)
        assert np.array_equal(held, refs)
        if info == 0:
            for i in range(R):
                if lens[i] > old[i] and old[i] % page:
                    assert refs[table[i][old[i] // page]] == 1  # its own to write
                assert (src[i] >= 0) == (lens[i] > old[i] and old[i] % page > 0
                                         and table[i][old[i] // page] != before[i][old[i] // page])
        nt, nr, s, d, L = blocks.compact(table, refs)
        assert sorted(nr[:L]) == sorted(n for n in refs if n) and not any(nr[L:])
        assert all(x >= L > y for x, y in zip(s, d))
        content = {p: p for p in range(60)}
        content.update(zip(d, s))
        assert [[content[p] if p >= 0 else -1 for p in r] for r in nt] == table
        table, refs = nt, nr


def test_verified_tokens_have_the_targets_law():
    """Every pair of random numbers on a fine grid, every drafted token: p, to the grid's step."""
    rng = np.random.default_rng(3)
    V, n = 4, 40
    for point in (False, True):
        tx, dx = rng.normal(size=V), rng.normal(size=V)
        p, q = blocks.softmax(tx, 1.0), blocks.softmax(dx, 1.0)
        got = np.zeros(V)
        law = np.eye(V)[2] if point else q
        for x in range(V):
            if law[x] == 0:
                continue
            for u in (np.arange(n) + 0.5) / n:
                for un in (np.arange(n) + 0.5) / n:
                    a, t, lp, _ = blocks.verify(np.stack([tx, tx]), None if point else np.stack([dx, dx]), [x, 0], [0, 2], [u, u], [un])
                    got[t[0]] += law[x] / n ** 2
                    assert np.isclose(lp[0], np.log(p[t[0]]))
        assert np.all(np.abs(got - p) <= 2.0 / n)


def test_greedy_verification():
    x = np.array([[0.0, 3.0, 3.0], [1.0, 0.0, 5.0], [9.0, 0.0, 0.0]])
    a, t, lp, _ = blocks.verify(x, None, [1, 2, 7], [0, 3], [0.9] * 3, [0.5], [0.0])
    assert a[0] == 2 and list(t) == [1, 2, 0] and not lp.any()
    a, t, _, _ = blocks.verify(x, None, [2, 2, 7], [0, 3], [0.0] * 3, [0.5], [0.0])
    assert a[0] == 0 and list(t) == [1, -1, -1]
