"""GPU: token log probabilities, entropy and top alternatives against fp64.

Bounds.  With d = x - m (exact to half a step of the larger operand: e^d is off by
|d| 2^-24 + a few steps of exp, under 2^-19 for |d| <= 16 and weighted by e^d
beyond), the sums of at most V terms grow pairwise in a lane's chain of V / 2048
chunks and a tree: relative error of r and t under 2^-18 for the sizes here.
log p is then off by 2^-18 r / (1 + r) <= 2^-18, and by half a step of x - m; the
entropy by 2^-18 (1 + |t| / (1 + r)) and the step of its two terms."""
import numpy as np
import pytest

from oracle import lowp

from gpu_util import host, need_gpu, say, torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _run(q, x, ids, top, **kw):
    T = x.shape[0]
    lp, ent = torch.full((T,), 9.0, device="cuda"), torch.full((T,), 9.0, device="cuda")
    ti = torch.full((T, top), -7, dtype=torch.int32, device="cuda")
    tl = torch.full((T, top), 9.0, device="cuda")
    q.token_logprobs(x, ids, lp, ent, ti, tl, **kw)
    return lp, ent, ti, tl


def _close(got, want, tol):
    got, want = np.asarray(got, float), np.asarray(want, float)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])
    bad = np.abs(got[fin] - want[fin]) - tol * (1 + np.abs(want[fin]))
    assert bad.size == 0 or bad.max() <= 0, bad.max()


def _check(q, x, ids, top, tol=2.0 ** -18):
    """x: host tensor of the logits' type."""
    xd = x.cuda()
    got = _run(q, xd, None if ids is None else torch.from_numpy(ids).cuda(), top) \
        if ids is not None else None
    lp, ent, ti, tl = lowp.logprobs(x.double().numpy(), ids, top)
    assert np.array_equal(host(got[2]), ti)
    _close(host(got[0]), lp, tol)
    _close(host(got[1]), ent, tol)
    _close(host(got[3]), tl, tol)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,top", [(1, 1, 1), (1, 2, 0), (3, 7, 7), (2, 31, 20), (5, 100, 32),
                                     (4, 2047, 5), (2, 2049, 32), (1, 5000, 20), (2, 50257, 20),
                                     (300, 1000, 5), (257, 4099, 1), (600, 33, 32), (1, 131072, 32),
                                     (9, 32000, 5)])
def test_rows(T, V, top, dtype):
    q = need_gpu()
    rng = np.random.default_rng(T * 100003 + V)
    x = torch.from_numpy(rng.normal(size=(T, V)) * 3).to(DT[dtype])
    ids = rng.integers(0, V, size=T)
    say("logprobs", T, V, top, dtype)
    _check(q, x, ids, top)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 6000, 40000])
def test_masks_ties_and_special_rows(V, dtype):
    q = need_gpu()
    rng = np.random.default_rng(V)
    T = 14
    x = torch.from_numpy(rng.normal(size=(T, V)) * 3).to(DT[dtype])
    low = torch.finfo(DT[dtype]).min
    x[1] = -np.inf                       # nothing left
    x[2, 5:] = -np.inf                   # few left
    x[3] = 2.5                           # all equal
    x[4] = low                           # all at the type's lowest value
    x[5, : V // 2] = low                 # masked by it
    x[6, V // 3] = float("nan")
    x[7, V // 3] = float("inf")
    x[8] = torch.round(x[8])             # many ties
    x[9, 1:] = -np.inf                   # one left: certain
    x[9, 0] = -3.0
    x[10, V - 1] = 60.0                  # almost certain
    x[11] = 0.0
    x[11, ::2] = -0.0                    # both zeros are equal
    x[12] = float("nan")
    x[13, V // 2] = float("-inf")
    ids = rng.integers(0, V, size=T)
    ids[[0, 5, 9, 10, 13]] = [-1, V - 1, 0, V - 1, V // 2]
    ids[8] = V + 3                       # past the vocabulary
    say("logprobs, special rows", V, dtype)
    _check(q, x, ids, min(20, V))


def test_almost_certain_tokens_keep_their_digits():
    """log p of a certain token is -r, not log of a sum near 1."""
    q = need_gpu()
    x = torch.zeros((1, 1000))
    x[0, 7] = 25.0
    lp, ent, _, _ = _run(q, x.cuda(), torch.tensor([7], device="cuda"), 1)
    r = 999 * np.exp(-25.0)
    # e^-25 is off by 25 * 2^-24 and a few steps, its sum by 2^-18: 2^-17 relative
    assert abs(float(lp) + np.log1p(r)) <= 2.0 ** -17 * r
    want = np.log1p(r) + 25 * r / (1 + r)
    assert abs(float(ent) - want) <= 2.0 ** -17 * want


@pytest.mark.parametrize("T", [2, 300])
def test_candidates_beyond_the_list(T):
    """Every large logit in the same few lanes' share: more candidates than the list
    holds, the alternatives are taken one after another."""
    q = need_gpu()
    V = 262144
    rng = np.random.default_rng(4)
    x = torch.full((T, V), -20.0)
    lanes = (torch.arange(V) // 8) % 256 < 9
    x[:, lanes] = torch.from_numpy(rng.normal(size=(1, int(lanes.sum())))).float() + 5.0
    rows = [0, T - 1]
    say("logprobs, few lanes", T)
    got = _run(q, x.cuda(), torch.zeros(T, dtype=torch.int64, device="cuda"), 32)
    _, _, ti, tl = lowp.logprobs(x[rows].double().numpy(), None, 32)
    assert np.array_equal(host(got[2])[rows], ti)
    _close(host(got[3])[rows], tl, 2.0 ** -18)


def test_optional_outputs_strides_and_alignment():
    q = need_gpu()
    rng = np.random.default_rng(6)
    big = torch.from_numpy(rng.normal(size=(9, 3011)) * 2).float().cuda()
    ids = torch.from_numpy(rng.integers(0, 2999, size=9)).cuda()
    for off in (0, 1, 4):
        x = big[:, off:off + 2999]
        full = _run(q, x, ids, 6)
        want = lowp.logprobs(host(x).astype(float), host(ids), 6)
        assert np.array_equal(host(full[2]), want[2])
        _close(host(full[0]), want[0], 2.0 ** -18)
        lp = torch.empty(9, device="cuda")
        q.token_logprobs(x, ids, lp)
        assert torch.equal(lp, full[0])
        ent = torch.empty(9, device="cuda")
        q.token_logprobs(x, None, None, ent)
        assert torch.equal(ent, full[1])
        ti, tl = torch.empty((9, 6), dtype=torch.int32, device="cuda"), torch.empty((9, 6), device="cuda")
        q.token_logprobs(x, None, None, None, ti, tl)
        assert torch.equal(ti, full[2]) and torch.equal(tl, full[3])
    # every other row
    got = _run(q, big[::2], ids[::2].contiguous(), 3)
    want = lowp.logprobs(host(big[::2]).astype(float), host(ids[::2]), 3)
    assert np.array_equal(host(got[2]), want[2])
    _run(q, big[:0], ids[:0], 3)  # no rows


def test_logits_past_32_bits():
    q = need_gpu()
    T, V = 40000, 60000  # 4.8 GB
    x = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    x[-1, -1], x[-2, 3] = 5.0, 4.0
    ids = torch.full((T,), V - 1, device="cuda")
    say("logprobs past 32 bits")
    lp, ent, ti, tl = _run(q, x, ids, 2)
    assert ti[-1].tolist() == [V - 1, 0] and ti[-2].tolist() == [3, 0] and ti[0].tolist() == [0, 1]
    want = 5 - np.log(V - 1 + np.exp(5.0))
    assert abs(float(lp[-1]) - want) <= 2.0 ** -18 * (1 + abs(want))


def test_captured_replayed_and_repeatable():
    q = need_gpu()
    x = torch.zeros((3, 70000), device="cuda")
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    outs = [torch.empty(3, device="cuda"), torch.empty(3, device="cuda"),
            torch.empty((3, 20), dtype=torch.int32, device="cuda"), torch.empty((3, 20), device="cuda")]
    q.token_logprobs(x, ids, *outs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.token_logprobs(x, ids, *outs)
    for turn in range(4):
        x.copy_(torch.randn(x.shape).to(torch.bfloat16))
        ids.copy_(torch.randint(0, 70000, (3,)))
        g.replay()
        torch.cuda.synchronize()
        want = _run(q, x, ids, 20)
        again = _run(q, x, ids, 20)
        for a, b, c in zip(outs, want, again):
            assert torch.equal(a, b) and torch.equal(b, c), turn
