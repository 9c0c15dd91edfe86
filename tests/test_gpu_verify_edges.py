"""GPU: calls of verify_drafts at the ends of what its header allows."""
import ctypes

import numpy as np
import pytest

from block_util import ints
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
