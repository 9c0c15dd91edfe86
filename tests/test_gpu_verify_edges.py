"""GPU: calls of verify_drafts at the ends of what its header allows."""
import ctypes

import numpy as np
import pytest

from oracle import blocks

from block_util import DT, ints
from gpu_util import host, need_gpu, say, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [10, 50000])
@pytest.mark.parametrize("temps", [False, True])
def test_sequences_without_rows(vocab, temps):
    """No rows: nothing but accepted is written, and no other array is needed."""
    q = need_gpu()
    S = 5
    acc, starts = ints([77] * S), ints([0] * (S + 1))
    t = torch.ones(S, device="cuda") if temps else None
    ws = torch.zeros(max(q.verify_drafts_workspace_size(0, vocab, S), 16), dtype=torch.uint8, device="cuda")
    say("verify, no rows", vocab, temps)
    status = q._lib.load().verify_drafts(None, 1, vocab, None, 0, 0, 0, vocab, None, starts.data_ptr(), S, None, None,
                                         t.data_ptr() if temps else None, acc.data_ptr(), None, None, ws.data_ptr(), ws.numel(),
                                         ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert status == 0
    torch.cuda.synchronize()
    assert np.all(host(acc) == 0)
    # the binding, whose arrays are there but empty
    acc.fill_(77)
    e = torch.empty(0, device="cuda")
    for draft in (torch.empty((0, vocab), device="cuda"), None):
        q.verify_drafts(torch.empty((0, vocab), device="cuda"), draft, torch.empty(0, dtype=torch.int64, device="cuda"), starts, e,
                        torch.zeros(S, device="cuda"), acc, torch.empty(0, dtype=torch.int64, device="cuda"), temperatures=t)
        torch.cuda.synchronize()
        assert np.all(host(acc) == 0)


def _same_as_the_oracle(q, target, draft, ids, starts, u, un, temps):
    f = lambda x: None if x is None else x.double().numpy()  # noqa: E731
    acc, tok, lp, margin = blocks.verify(f(target), f(draft), ids, starts, u.astype(float), un.astype(float), temps)
    assert margin > 2.0 ** -12, "a decision on its border"
    T, S = target.shape[0], len(starts) - 1
    ga, gt, gl = ints([77] * S), torch.full((T,), 77, dtype=torch.int64, device="cuda"), torch.full((T,), 77.0, device="cuda")
    d = lambda x: None if x is None else torch.as_tensor(x).cuda()  # noqa: E731
    q.verify_drafts(d(target), d(draft), d(ids), ints(starts), d(u), d(un), ga, gt, logprobs=gl,
                    temperatures=d(np.asarray(temps, dtype=np.float32)))
    torch.cuda.synchronize()
    assert np.array_equal(host(ga), acc)
    assert np.array_equal(host(gt), tok)
    assert np.all(np.abs(host(gl) - lp) <= 2.0 ** -18 * (1 + np.abs(lp)))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [70, 3000, 70000])
def test_logits_farther_apart_than_fp32_reaches(vocab, dt):
    """Masks of the type's lowest value beside a logit near its largest: their difference is no finite number.  The
    largest counts all the same, at temperature 0 as at others."""
    q = need_gpu()
    rng = np.random.default_rng(vocab)
    S = 4
    info = torch.finfo(DT[dt])
    target = torch.full((2 * S, vocab), info.min, dtype=DT[dt])
    ids = rng.integers(0, vocab, size=2 * S).astype(np.int64)
    target[torch.arange(2 * S), torch.from_numpy(ids)] = info.max
    target[2, ids[2]] = info.min
    target[2, (int(ids[2]) + vocab // 2) % vocab] = info.max  # a refusal
    u, un = np.full(2 * S, 0.5, np.float32), np.full(S, 0.5, np.float32)
    say("verify, far logits", vocab, dt)
    for temps in ([0.0] * S, [1.0, 0.0, 0.5, 2.0]):
        _same_as_the_oracle(q, target, None, ids, list(range(0, 2 * S + 1, 2)), u, un, temps)


@pytest.mark.parametrize("tiny", [1e-37, 5e-39, 4e-39, 1e-42, 1e-45])
def test_the_smallest_temperatures(tiny):
    """Towards 0 the law becomes the largest logit's (or that of those that tie for it); the reciprocal of a temperature
    below 2^-128 is no finite number."""
    q = need_gpu()
    rng = np.random.default_rng(5)
    S, vocab = 6, 2000
    target, draft = (torch.from_numpy(rng.normal(size=(2 * S, vocab))).float() for _ in range(2))
    ids = draft.argmax(1).numpy().astype(np.int64)
    ids[0::4] = target[0::4].argmax(1).numpy()
    draft[torch.arange(2 * S), torch.from_numpy(ids)] = 9.0
    target[3, :2] = target[3, 1990] = 50.0  # three tie
    target[6, -500:] = -np.inf
    u, un = np.full(2 * S, 0.5, np.float32), np.full(S, 0.5, np.float32)
    say("verify, tiny temperatures", tiny)
    temps = np.full(S, tiny, np.float32).astype(np.float64)
    for d in (draft, None):
        _same_as_the_oracle(q, target, d, ids, list(range(0, 2 * S + 1, 2)), u, un, temps)
