"""GPU: the sums of token_logprobs over long rows of nearly equal logits, where each
rounding of a running sum goes the same way.

A row has its maximum, 0, once in each lane's first chunk and v elsewhere: a lane adds
V / 256 - 1 equal terms.  e^v is off by (|v| + |v| / 2 + 1) 2^-24 <= 10 2^-24 (its
exponent's product, the constant, the instruction), a chunk's tree by 3, the
compensated chain by 2, the joins of 256 lanes by 11 half steps: 26 2^-24 of r.  Then
log p is off by that, 2 steps of log1p and half a step of the result; the entropy's
second term has twice that of r and the products' roundings."""
import numpy as np
import pytest

from gpu_util import host, need_gpu, say, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V", [(260, 262144), (256, 128000), (256, 1 << 20), (1, 1 << 20)])
def test_equal_terms(T, V, dtype):
    q = need_gpu()
    v = torch.linspace(-6.0, -0.05, T).to(dtype)
    x = v.cuda()[:, None].expand(T, V).contiguous()
    x[:, 0:2048:8] = 0
    ids = torch.full((T,), V - 1, device="cuda")
    lp, ent = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    say("logprobs, equal terms", T, V, dtype)
    q.token_logprobs(x, ids, lp, ent)
    v = v.double().numpy()
    r = 255 + (V - 256) * np.exp(v)
    second = (V - 256) * np.exp(v) * v / (1 + r)
    want, want_ent = v - np.log1p(r), np.log1p(r) - second
    tol = (26 + 2 * np.log1p(r) + np.abs(want)) * 2.0 ** -24
    assert np.all(np.abs(host(lp) - want) <= tol)
    tol = (26 + 2 * np.log1p(r) + 60 * np.abs(second) + want_ent) * 2.0 ** -24
    assert np.all(np.abs(host(ent) - want_ent) <= tol)
