"""GPU: drafted tokens against the target's logits.  Tokens have to be the oracle's: each case's
closest decision is checked (on the CPU) to be farther from its border than the sums' error, fp32's for an acceptance
(2^-19 of the ratio: a sum of up to 2^18 terms in trees, exponentials of |x - m| up to 30), fp64's for a
draw."""
import numpy as np
import pytest

from oracle import blocks

from block_util import DT, ints, starts_of
from gpu_util import host, need_gpu, say, torch

pytestmark = pytest.mark.gpu


def _case(rng, counts, V, point=False, masked=0, spread=2.5):
    T = sum(counts)
    base = rng.normal(size=(T, V)) * spread
    target = torch.from_numpy(base + 0.5 * rng.normal(size=(T, V)))
    draft = torch.from_numpy(base + 0.5 * rng.normal(size=(T, V)))
    if masked:
        target[:, V - masked:] = draft[:, V - masked:] = -np.inf
    ids = np.array([rng.choice(V, p=_p(draft[t].numpy())) if not point else int(draft[t].argmax()) for t in range(T)], dtype=np.int64)
    return target, draft, ids, rng.random(T).astype(np.float32), rng.random(len(counts)).astype(np.float32)


def _p(x):
    e = np.exp(x - x.max())
    return e / e.sum()


def _run(q, target, draft, ids, starts, u, u_next, temps=None, pad=0):
    T = target.shape[0]
    tokens = torch.full((T,), 77, dtype=torch.int64, device="cuda")
    lp = torch.full((T,), 77.0, device="cuda")
    acc = ints([77] * (len(starts) - 1))
    d = lambda x: None if x is None else torch.as_tensor(x).cuda()  # noqa: E731
    q.verify_drafts(target.cuda(), None if draft is None else draft.cuda(), d(ids), ints(starts), d(u), d(u_next), acc, tokens,
                    logprobs=lp, temperatures=None if temps is None else d(np.asarray(temps, dtype=np.float32)))
    torch.cuda.synchronize()
    return host(acc), host(tokens), host(lp)


def _check(q, target, draft, ids, starts, u, u_next, temps=None):
    f = lambda x: None if x is None else x.double().numpy()  # noqa: E731
    acc, tok, lp, margin = blocks.verify(f(target), f(draft), ids, starts, u.astype(float), u_next.astype(float), temps)
    assert margin > 1e-9, "a decision on its border"
    ga, gt, gl = _run(q, target, draft, ids, starts, u, u_next, temps)
    n = starts[-1]
    assert np.array_equal(ga, acc)
    assert np.array_equal(gt[:n], tok[:n]) and np.all(gt[n:] == 77) and np.all(gl[n:] == 77)
    assert np.all(np.abs(gl[:n] - lp[:n]) <= 2.0 ** -18 * (1 + np.abs(lp[:n])))
    return acc


@pytest.mark.parametrize("point", [False, True])
@pytest.mark.parametrize("counts,V,tdt,ddt,masked,temps", [
    ([1], 2, "f32", "f32", 0, None),
    ([5, 5, 5], 1000, "bf16", "bf16", 20, None),
    ([1, 4, 2, 9, 3], 4099, "f32", "bf16", 0, [1.0, 0.7, 0.0, 1.5, 0.0]),
    ([3] * 40, 257, "bf16", "f32", 7, None),
    ([4, 0, 2], 50257, "bf16", "bf16", 100, None),
    ([6, 3], 128000, "f32", "f32", 0, [0.9, 1.0]),
    ([70], 33, "f32", "f32", 0, None),
])
def test_verify(point, counts, V, tdt, ddt, masked, temps):
    q = need_gpu()
    rng = np.random.default_rng(V + len(counts))
    target, draft, ids, u, u_next = _case(rng, counts, V, point, masked)
    target, draft = target.to(DT[tdt]), draft.to(DT[ddt])
    say("verify", point, counts, V, tdt, ddt, temps)
    _check(q, target, None if point else draft, ids, starts_of(counts), u, u_next, temps)
    # padding behind the last sequence
    if len(counts) > 2 and counts[-1]:
        _check(q, target, None if point else draft, ids, starts_of(counts[:-1]), u, u_next[:-1],
               None if temps is None else temps[:-1])


def test_strided_rows():
    """Rows of a larger matrix, which start off any border."""
    q = need_gpu()
    rng = np.random.default_rng(31)
    target, draft, ids, u, u_next = _case(rng, [4, 4], 1001)
    for dt in (torch.bfloat16, torch.float32):
        wt, wd = (torch.full((8, 1013), 50.0, dtype=dt) for _ in range(2))
        wt[:, 5:1006], wd[:, 7:1008] = target.to(dt), draft.to(dt)
        acc, tok, lp, _ = blocks.verify(wt[:, 5:1006].double().numpy(), wd[:, 7:1008].double().numpy(), ids, [0, 4, 8],
                                        u.astype(float), u_next.astype(float))
        a, t, p = ints([0, 0]), torch.zeros(8, dtype=torch.int64, device="cuda"), torch.zeros(8, device="cuda")
        say("verify strided", dt)
        q.verify_drafts(wt.cuda()[:, 5:1006], wd.cuda()[:, 7:1008], torch.from_numpy(ids).cuda(), ints([0, 4, 8]),
                        torch.from_numpy(u).cuda(), torch.from_numpy(u_next).cuda(), a, t, logprobs=p)
        assert np.array_equal(host(a), acc) and np.array_equal(host(t), tok)


def test_sure_refusals_and_acceptances():
    """u = 0 accepts whatever the target allows; a token that it rules out is never accepted; equal
    laws accept everything; the draw behind a refusal never gives what only the drafter likes."""
    q = need_gpu()
    V, S = 300, 6
    rng = np.random.default_rng(32)
    x = torch.from_numpy(rng.normal(size=(2 * S, V))).float()
    ids = rng.integers(0, V, size=2 * S).astype(np.int64)
    starts = starts_of([2] * S)
    u, un = np.full(2 * S, 0.999, np.float32), rng.random(S).astype(np.float32)
    say("verify sure")
    a, t, _ = _run(q, x, x, ids, starts, u, un)
    assert np.all(a == 1) and np.array_equal(t[0::2], ids[0::2]) and np.all(t[1::2] >= 0)
    y = x.clone()
    y[np.arange(2 * S), ids] = -np.inf
    a, t, lp = _run(q, y, x, ids, starts, np.zeros(2 * S, np.float32), un)
    assert np.all(a == 0) and np.all(t[0::2] != ids[0::2]) and np.all(t[1::2] == -1) and np.all(lp[1::2] == 0)
    a, t, _ = _run(q, y, None, ids, starts, np.zeros(2 * S, np.float32), un)
    assert np.all(a == 0) and np.all(t[0::2] != ids[0::2])
    # the first and last border of the draw
    a, t, _ = _run(q, x[:1], None, ids[:1], [0, 1], u[:1], np.zeros(1, np.float32))
    assert t[0] == 0
    a, t, _ = _run(q, x[:1], None, ids[:1], [0, 1], u[:1], np.full(1, np.nextafter(np.float32(1), np.float32(0))))
    assert t[0] == V - 1
    z = x[:1].clone()
    z[0, :10] = z[0, 200:] = -np.inf
    for un_, want in ((0.0, 10), (np.nextafter(np.float32(1), np.float32(0)), 199), (2.0, 199), (float("nan"), 10), (-1.0, 10)):
        assert _run(q, z, None, ids[:1], [0, 1], u[:1], np.full(1, un_, np.float32))[1][0] == want


@pytest.mark.parametrize("temps", [None, [0.0] * 8])
def test_rows_that_are_no_law(temps):
    """NaN, +inf, nothing but -inf, ids outside the vocabulary."""
    q = need_gpu()
    rng = np.random.default_rng(33)
    V, S = 500, 8
    target, draft, ids, u, un = _case(rng, [3] * S, V)
    target, draft = target.float(), draft.float()
    ids[0::3] = target[0::3].argmax(1)
    u[:] = 0.0
    target[0, 7] = float("nan")
    target[3, 7] = float("inf")
    target[6] = -np.inf
    draft[9, 3] = float("nan")
    draft[12] = -np.inf
    ids[15], ids[18] = -5, V
    target[22] = -np.inf  # behind an accepted token
    say("verify no law", temps)
    a, t, lp = _run(q, target, draft, ids, starts_of([3] * S), u, un, temps)
    assert np.all(a[:3] == 0) and np.all(t[:9] == -1) and np.all(lp[:9] == 0)
    if temps is None:
        assert np.all(a[3:7] == 0) and np.all(t[9:21:3] >= 0)
    else:
        assert np.all(a[3:5] >= 1) and np.all(a[5:7] == 0)
        assert np.array_equal(t[15:21:3], host(target[15:21:3].argmax(1)))
    assert a[7] == 1 and t[21] == ids[21] and t[22] == -1


def test_frequencies():
    """Over a grid of both random numbers, the tokens have the target's probabilities."""
    q = need_gpu()
    rng = np.random.default_rng(34)
    V, n = 5, 64
    tx, dx = rng.normal(size=V), rng.normal(size=V)
    p, d = _p(tx), _p(dx)
    S = n * n
    target = torch.from_numpy(np.tile(tx, (2 * S, 1))).float()
    draft = torch.from_numpy(np.tile(dx, (2 * S, 1))).float()
    grid = ((np.arange(n) + 0.5) / n).astype(np.float32)
    u = np.zeros(2 * S, np.float32)
    u[0::2] = np.repeat(grid, n)
    un = np.tile(grid, n)
    got = np.zeros(V)
    say("verify frequencies")
    for x in range(V):
        ids = np.full(2 * S, x, np.int64)
        t = _run(q, target, draft, ids, starts_of([2] * S), u, un)[1]
        got += d[x] * np.bincount(t[0::2], minlength=V) / S
    # a border of either number moves by less than a cell: 1 / n each
    assert np.all(np.abs(got - p) <= 2.0 / n)


def test_many_sequences():
    q = need_gpu()
    rng = np.random.default_rng(35)
    counts = [int(v) for v in rng.integers(0, 4, size=700)]
    target, draft, ids, u, un = _case(rng, counts, 64)
    say("verify many")
    _check(q, target.float(), draft.float(), ids, starts_of(counts), u, un)


def test_captured_and_replayed():
    q = need_gpu()
    rng = np.random.default_rng(36)
    counts, V = [5, 3, 4], 40000
    T, st = sum(counts), ints(starts_of(counts))
    target, draft = (torch.zeros((T, V), device="cuda") for _ in range(2))
    ids = torch.zeros(T, dtype=torch.int64, device="cuda")
    u, un, temps = torch.zeros(T, device="cuda"), torch.zeros(3, device="cuda"), torch.ones(3, device="cuda")
    outs = [[ints([0] * 3), torch.zeros(T, dtype=torch.int64, device="cuda"), torch.zeros(T, device="cuda")] for _ in range(2)]

    def step(o):
        q.verify_drafts(target, draft, ids, st, u, un, *o[:2], logprobs=o[2], temperatures=temps)

    step(outs[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(outs[0])
    for turn in range(4):
        a, b, i, uu, nn = _case(rng, counts, V)
        for t, v in ((target, a), (draft, b), (ids, torch.from_numpy(i)), (u, torch.from_numpy(uu)), (un, torch.from_numpy(nn))):
            t.copy_(v)
        temps.copy_(torch.tensor([1.0, 0.0, 0.8]))
        g.replay()
        torch.cuda.synchronize()
        step(outs[1])
        torch.cuda.synchronize()
        for x, y in zip(*outs):
            assert torch.equal(x, y), turn


def test_the_binding_refuses():
    q = need_gpu()
    x = torch.zeros((3, 10), device="cuda")
    i, s = torch.zeros(3, dtype=torch.int64, device="cuda"), ints([0, 3])
    u, un, a, t = torch.zeros(3, device="cuda"), torch.zeros(1, device="cuda"), ints([0]), torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (lambda: q.verify_drafts(x, x[:2], i, s, u, un, a, t),
                lambda: q.verify_drafts(x, x[:, :9], i, s, u, un, a, t),
                lambda: q.verify_drafts(x, x, i[:2], s, u, un, a, t),
                lambda: q.verify_drafts(x, x, i, s, u[:2], un, a, t),
                lambda: q.verify_drafts(x, x, i, s.cpu(), u, un, a, t),
                lambda: q.verify_drafts(x[0], x, i, s, u, un, a, t)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q.verify_drafts(x.half(), x, i, s, u, un, a, t),
                lambda: q.verify_drafts(x, x, i.int(), s, u, un, a, t),
                lambda: q.verify_drafts(x, x, i, s, u, un, a, t.int())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(q.GPTQError):
        q.verify_drafts(x, x, i, s, u, un, a, i)
