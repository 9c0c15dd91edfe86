"""GPU: a cache of one page with more than 2^30 slots, its last slots written and read."""
import numpy as np
import pytest

from oracle import lowp

from gpu_util import host, need_gpu, say, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [6, 1100])
def test_more_than_2_30_slots_in_a_page(tokens):
    q = need_gpu()
    page, D = 2 ** 30 + 9, 16
    codes = torch.zeros((1, page, 1, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((1, page, 1, 1), device="cuda")
    c = q.make_kv_cache(codes, scales, None, D, "int4", 16)
    slots = torch.arange(page - tokens + 2, page + 2, device="cuda")
    slots[-2:] = torch.tensor([0, -1])
    x = torch.randn((tokens, 1, D), generator=torch.Generator().manual_seed(1)).cuda()
    back = torch.full_like(x, 7.0)
    say("cache of one page", page, tokens)
    q.kv_cache_write(x, None, slots, c, None)
    q.kv_cache_read(c, None, slots, back, None)
    rows = host(x)[:, 0].astype(float)
    want = lowp.kv_dequantize(*lowp.kv_quantize(rows, "int4", 16, False), "int4", 16)
    want[-1] = 0
    # (q - 8) s in fp32: half a step
    assert np.all(np.abs(host(back)[:, 0] - want) <= 2.0 ** -24 * np.abs(want))
    assert int(torch.count_nonzero(scales[0, 1:page - tokens + 2])) == 0
