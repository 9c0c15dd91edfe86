"""How near the decisions of the cases in test_gpu_verify come to their borders: acceptances apart from draws, each
against the error that its arithmetic allows.

An acceptance compares u q(x) with p(x), both fp32.  Each is e^-d over a sum, d = (m - x) / temperature.  d has four roundings
(the difference, log2 e, its quotient by the temperature, the product), so e^-d is off by 4 d 2^-24, and the sum by the mean of
4 d 2^-24 under the law itself: at most 4 ln(vocab) 2^-24, since that mean is the law's entropy less the logarithm of the sum,
which is 1 or more.  The exponentials, their rescaling when a maximum moves, the sums in trees, the joins of lanes, waves and
segments and the quotient are some 64 roundings more at the very most."""
import math

import numpy as np
import pytest

from oracle import blocks

from block_util import DT, starts_of
from gpu_util import torch
import test_gpu_verify as cases

CASES = next(m.args[1] for m in cases.test_verify.pytestmark if m.name == "parametrize" and m.args[0] != "point")


def _far_enough(target, draft, ids, starts, u, un, temps=None):
    f = lambda x: None if x is None else x.double().numpy()  # noqa: E731
    args = f(target), f(draft), ids, starts, u.astype(float), un.astype(float), temps
    *out, accepts, draws = blocks.verify_margins(*args)
    models, V = 1 if draft is None else 2, target.shape[1]
    for margin, below in accepts:
        assert margin > 8 * (4 * (below + models * math.log(V)) + 64 * models) * 2.0 ** -24
    assert draws > 1e-9
    # the one number that both make
    want = blocks.verify(*args)
    assert all(np.array_equal(a, b) for a, b in zip(out, want)) and want[3] == min([m for m, _ in accepts] + [draws])


@pytest.mark.parametrize("point", [False, True])
@pytest.mark.parametrize("counts,V,tdt,ddt,masked,temps", CASES)
def test_verify(point, counts, V, tdt, ddt, masked, temps):
    target, draft, ids, u, un = cases._case(np.random.default_rng(V + len(counts)), counts, V, point, masked)
    _far_enough(target.to(DT[tdt]), None if point else draft.to(DT[ddt]), ids, starts_of(counts), u, un, temps)


def test_strided_rows_and_many_sequences():
    target, draft, ids, u, un = cases._case(np.random.default_rng(31), [4, 4], 1001)
    for dt in (torch.bfloat16, torch.float32):
        _far_enough(target.to(dt), draft.to(dt), ids, [0, 4, 8], u, un)
    rng = np.random.default_rng(35)
    counts = [int(v) for v in rng.integers(0, 4, size=700)]
    target, draft, ids, u, un = cases._case(rng, counts, 64)
    _far_enough(target.float(), draft.float(), ids, starts_of(counts), u, un)


def test_a_decision_near_its_border_is_seen():
    x = torch.zeros((2, 4))
    with pytest.raises(AssertionError):  # p = 1/4, and u a last place off it
        _far_enough(x, None, np.array([1, 0]), [0, 2], np.array([np.nextafter(np.float32(0.25), np.float32(1)), 0], np.float32),
                    np.array([0.4], np.float32))
