"""GPU: the quantized key/value cache against the fp64 oracle.  What is written
(codes, scales, zeros) has to be equal bit for bit; what is read is
(q - zero) * scale with one fp32 rounding of the product and one to the output's
type: within half a step of 2^-24 and of the type."""
import numpy as np
import pytest

import oracle
from oracle import lowp

from gpu_util import host, need_gpu, say, torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Cache:
    """A cache of known contents, in a page order of choice."""

    def __init__(self, q, pages, page, heads, dim, fmt, group, asym, order="phd"):
        nb = dim // 2 if fmt == "int4" else dim
        ng = 1 if group <= 0 else -(-dim // group)
        if order == "phd":  # [pages, page, heads, bytes]
            self.codes = torch.full((pages, page, heads, nb), 0x55, dtype=torch.uint8, device="cuda")
            self.scales = torch.full((pages, page, heads, ng), -1.0, device="cuda")
            self.zeros = torch.full((pages, page, heads, ng), 99, dtype=torch.uint8, device="cuda")
        else:  # heads before the page's slots, rows padded
            self.codes = torch.full((pages, heads, page, nb + 8), 0x55, dtype=torch.uint8,
                                    device="cuda")[..., :nb].transpose(1, 2)
            self.scales = torch.full((pages, heads, page, ng + 1), -1.0, device="cuda")[..., :ng].transpose(1, 2)
            self.zeros = torch.full((pages, heads, page, ng + 1), 99, dtype=torch.uint8,
                                    device="cuda")[..., :ng].transpose(1, 2)
        self.fmt, self.group, self.asym, self.dim, self.page = fmt, group, asym, dim, page
        self.h = q.make_kv_cache(self.codes, self.scales, self.zeros if asym else None, dim, fmt, group)

    def flat(self):
        return [host(t).reshape(-1, *t.shape[2:]) for t in (self.codes, self.scales, self.zeros)]


def _check_written(c, x, slots):
    """The last row of each slot is there; every other slot is as it was."""
    codes, scales, zeros = c.flat()
    T, H, D = x.shape
    last = {int(s): t for t, s in enumerate(slots) if 0 <= s < codes.shape[0]}
    for s, t in last.items():
        qc, qs, qz = lowp.kv_quantize(x[t], c.fmt, c.group, c.asym)
        assert np.array_equal(codes[s], lowp.kv_pack(qc, c.fmt)), (s, t)
        assert np.array_equal(scales[s], qs.astype(np.float32)), (s, t)
        if c.asym:
            assert np.array_equal(zeros[s], qz.astype(np.uint8)), (s, t)
    rest = np.setdiff1d(np.arange(codes.shape[0]), list(last))
    assert np.all(codes[rest] == 0x55) and np.all(scales[rest] == -1) and np.all(zeros[rest] == 99)


def _check_read(c, slots, out, dtype):
    codes, scales, zeros = c.flat()
    D = c.dim
    got = host(out.double())
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for t, s in enumerate(slots):
        if not 0 <= s < codes.shape[0]:
            assert np.all(got[t] == 0)
            continue
        raw = codes[s]
        if c.fmt == "int4":
            raw = np.stack([raw & 15, raw >> 4], -1).reshape(raw.shape[0], D)
        z = zeros[s].astype(float) if c.asym else np.full(scales[s].shape, 8.0 if c.fmt == "int4" else 128.0)
        want = lowp.kv_dequantize(raw, scales[s].astype(float), z, c.fmt, c.group)
        assert np.all(np.abs(got[t] - want) <= (half + 2.0 ** -24 * (1 + half)) * np.abs(want)), t


FORMS = [("int8", True), ("int8", False), ("int4", True), ("int4", False), ("e4m3", False)]


@pytest.mark.parametrize("fmt,asym", FORMS)
@pytest.mark.parametrize("T,H,D,group,page,order,xdt,ydt", [
    (1, 1, 8, -1, 1, "phd", "bf16", "bf16"),
    (5, 2, 64, 64, 16, "phd", "bf16", "f32"),
    (7, 3, 80, 32, 4, "hpd", "f32", "bf16"),
    (9, 8, 128, 128, 16, "phd", "bf16", "bf16"),
    (33, 1, 192, 128, 7, "hpd", "bf16", "bf16"),
    (20, 4, 256, 256, 16, "phd", "f32", "f32"),
    (6, 2, 512, -1, 2, "phd", "bf16", "bf16"),
    (3, 1, 1024, 512, 2, "hpd", "f32", "bf16"),
    (300, 1, 8, 16, 64, "phd", "f32", "f32"),
    (12, 2, 40, 16, 5, "phd", "bf16", "bf16"),
])
def test_write_and_read(fmt, asym, T, H, D, group, page, order, xdt, ydt):
    q = need_gpu()
    rng = np.random.default_rng(T * 131 + H * 17 + D)
    pages = -(-(2 * T + 3) // page)
    kc, vc = (Cache(q, pages, page, H, D, fmt, group, asym, order) for _ in range(2))
    kv = torch.from_numpy(rng.standard_t(4, size=(T, 3 * H, D)) * 5).to(DT[xdt])
    kv[0, H] = 0.0  # a row of zeros
    K, V = kv[:, H:2 * H], kv[:, 2 * H:]
    d = kv.cuda()
    slots = rng.permutation(pages * page)[:T]
    if T > 4:
        slots[[1, 3]] = -1
    sd = torch.from_numpy(slots).cuda()
    say("kv write", fmt, asym, T, H, D, group, page, order, xdt)
    q.kv_cache_write(d[:, H:2 * H], d[:, 2 * H:], sd, kc.h, vc.h)
    torch.cuda.synchronize()
    _check_written(kc, K.double().numpy(), slots)
    _check_written(vc, V.double().numpy(), slots)
    rd = np.concatenate([slots, slots[::-1], [-1]])
    Ko, Vo = (torch.full((len(rd), H, D + 8), 3.0, dtype=DT[ydt], device="cuda") for _ in range(2))
    say("kv read")
    q.kv_cache_read(kc.h, vc.h, torch.from_numpy(rd).cuda(), Ko[..., :D], Vo[..., :D])
    _check_read(kc, rd, Ko[..., :D], ydt)
    _check_read(vc, rd, Vo[..., :D], ydt)
    assert torch.all(Ko[..., D:] == 3) and torch.all(Vo[..., D:] == 3)


@pytest.mark.parametrize("page,order", [(16, "phd"), (16, "hpd"), (24, "hpd")])
@pytest.mark.parametrize("fmt,asym", FORMS)
def test_long_calls(fmt, asym, page, order):
    """Enough rows for several units a lane, heads that fill no wave: every row's codes
    against rtn_minmax's form of the oracle, whole arrays at once."""
    q = need_gpu()
    rng = np.random.default_rng(page)
    T, H, D, G = 6001, 3, 160, 64
    pages = -(-6100 // page)
    kc, vc = (Cache(q, pages, page, H, D, fmt, G, asym, order) for _ in range(2))
    K, V = (torch.from_numpy(rng.normal(size=(T, H, D))).to(torch.bfloat16) for _ in range(2))
    slots = rng.permutation(pages * page)[:T]
    sd = torch.from_numpy(slots).cuda()
    say("kv long", fmt, asym, page, order)
    q.kv_cache_write(K.cuda(), V.cuda(), sd, kc.h, vc.h)
    Ko, Vo = (torch.empty((T, H, D), device="cuda") for _ in range(2))
    q.kv_cache_read(kc.h, vc.h, sd, Ko, Vo)
    for c, x, o in ((kc, K, Ko), (vc, V, Vo)):
        codes, scales, zeros = c.flat()
        qc, qs, qz = lowp.kv_quantize(x.double().numpy().reshape(T * H, D), fmt, G, asym)
        assert np.array_equal(codes[slots], lowp.kv_pack(qc, fmt).reshape(T, H, -1))
        assert np.array_equal(scales[slots], qs.astype(np.float32).reshape(T, H, -1))
        if asym:
            assert np.array_equal(zeros[slots], qz.astype(np.uint8).reshape(T, H, -1))
        rest = np.setdiff1d(np.arange(codes.shape[0]), slots)
        assert np.all(codes[rest] == 0x55) and np.all(scales[rest] == -1)
        want = lowp.kv_dequantize(qc, qs, qz, fmt, G).reshape(T, H, D)
        assert np.all(np.abs(host(o) - want) <= 2.0 ** -23 * np.abs(want))


@pytest.mark.parametrize("fmt,asym", FORMS)
def test_integers_equal_rtn_minmax(fmt, asym):
    """The integer formats' grid is rtn_minmax's: the same codes, scales and zeros."""
    if fmt == "e4m3":
        pytest.skip("not an integer format")
    q = need_gpu()
    rng = np.random.default_rng(77)
    T, D, G = 64, 128, 64
    x = torch.from_numpy(rng.normal(size=(T, 1, D))).to(torch.bfloat16).cuda()
    x[3, 0] = torch.arange(D, device="cuda") / 16 - 4  # many quotients half way between codes
    c = Cache(q, 4, 16, 1, D, fmt, G, asym)
    q.kv_cache_write(x, None, torch.arange(T, device="cuda"), c.h, None)
    bits = 4 if fmt == "int4" else 8
    codes = torch.empty((T, D), dtype=torch.uint8, device="cuda")
    s, z = (torch.empty((T, D // G), device="cuda") for _ in range(2))
    q.rtn_minmax(x.view(T, D), bits, G, codes, s, z, sym=not asym)
    got = c.codes.view(T, -1)
    if fmt == "int4":
        got = torch.stack([got & 15, got >> 4], 2).view(T, D)
    assert torch.equal(got, codes) and torch.equal(c.scales.view(T, -1), s)
    if asym:
        assert torch.equal(c.zeros.view(T, -1).float(), z)


@pytest.mark.parametrize("T", [6, 700, 1024, 1025, 3000, 9000])
def test_repeated_slots_keep_the_last_row(T):
    q = need_gpu()
    rng = np.random.default_rng(T)
    H, D = 2, 64
    c = Cache(q, 16, 16, H, D, "int8", 64, True)
    slots = rng.integers(-2, 256 + 2, size=T)  # some padding, some past the end
    x = torch.from_numpy(rng.normal(size=(T, H, D))).to(torch.bfloat16)
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    say("kv repeated slots", T)
    q.kv_cache_write(x.cuda(), None, torch.from_numpy(slots).cuda(), c.h, None, info=info)
    torch.cuda.synchronize()
    _check_written(c, x.double().numpy(), np.where(slots < 0, -1, slots))
    assert int(info) == int((slots >= 256).any())
    out = torch.empty((T, H, D), device="cuda")
    info.zero_()
    q.kv_cache_read(c.h, None, torch.from_numpy(slots).cuda(), out, None, info=info)
    _check_read(c, slots, out, "f32")
    assert int(info) == int((slots >= 256).any())


def test_keys_and_values_of_different_shapes():
    q = need_gpu()
    rng = np.random.default_rng(9)
    T = 40
    kc = Cache(q, 3, 16, 1, 192, "e4m3", 64, False)
    vc = Cache(q, 3, 16, 2, 64, "int4", 32, True)
    K = torch.from_numpy(rng.normal(size=(T, 1, 192))).float()
    V = torch.from_numpy(rng.normal(size=(T, 2, 64))).float()
    slots = rng.permutation(48)[:T]
    sd = torch.from_numpy(slots).cuda()
    say("kv of two shapes")
    q.kv_cache_write(K.cuda(), V.cuda(), sd, kc.h, vc.h)
    _check_written(kc, K.double().numpy(), slots)
    _check_written(vc, V.double().numpy(), slots)
    Ko, Vo = torch.empty((T, 1, 192), device="cuda"), torch.empty((T, 2, 64), device="cuda")
    q.kv_cache_read(kc.h, vc.h, sd, Ko, Vo)
    _check_read(kc, slots, Ko, "f32")
    _check_read(vc, slots, Vo, "f32")


def test_non_finite_rows():
    """A NaN takes code 0 of an integer group, an infinity gives its group an infinite
    scale, so that nothing finite is read from it ((q - zero) * inf); in e4m3 each non-finite value reads as NaN and nothing else does."""
    q = need_gpu()
    x = torch.linspace(-1, 1, 64).repeat(4, 1, 1)
    x[1, 0, 5], x[2, 0, 40], x[3, 0, 40] = float("nan"), float("inf"), float("-inf")
    sd = torch.arange(4, device="cuda")
    for fmt, asym in FORMS:
        c = Cache(q, 1, 4, 1, 64, fmt, 32, asym)
        say("kv non-finite", fmt, asym)
        q.kv_cache_write(x.cuda(), None, sd, c.h, None)
        out = torch.empty((4, 1, 64), device="cuda")
        q.kv_cache_read(c.h, None, sd, out, None)
        nan = host(torch.isnan(out) if fmt == "e4m3" else ~torch.isfinite(out))[:, 0]
        assert not nan[0].any()
        want = np.zeros((4, 64), bool)
        if fmt == "e4m3":
            want[1, 5] = want[2, 40] = want[3, 40] = True
        else:
            want[2:, 32:] = True
            codes = c.flat()[0][1, 0]
            assert (codes[2] >> 4 if fmt == "int4" else codes[5]) == 0
        assert np.array_equal(nan, want), (fmt, asym)


def test_codes_past_32_bits():
    """A cache of more than 2^32 bytes: its last slots are written and read."""
    q = need_gpu()
    pages, page, H, D = 40000, 64, 16, 128
    codes = torch.empty((pages, page, H, D), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((pages, page, H, 1), device="cuda")
    h = q.make_kv_cache(codes, scales, None, D, "int8", 128)
    n = pages * page
    slots = torch.tensor([n - 1, 5, n - 64, n // 2], device="cuda")
    x = torch.randn((4, H, D), device="cuda")
    say("kv past 32 bits", n)
    q.kv_cache_write(x, None, slots, h, None)
    out = torch.empty_like(x)
    q.kv_cache_read(h, None, slots, out, None)
    step = scales.view(n, H, 1)[slots]
    # half a step, and the fp32 roundings of quotient and product (2^-23 of 128 steps)
    assert torch.all((out - x).abs() <= step * (0.5 + 2.0 ** -15))
    assert torch.count_nonzero(scales) == 4 * H


def test_cache_captured_and_replayed():
    q = need_gpu()
    T, H, D = 9500, 2, 64
    c, e = (Cache(q, 600, 16, H, D, "int4", 32, True) for _ in range(2))
    x = torch.zeros((T, H, D), device="cuda")
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")
    out, want = torch.empty_like(x), torch.empty_like(x)

    def step(cache, o):
        q.kv_cache_write(x, None, slots, cache.h, None)
        q.kv_cache_read(cache.h, None, slots, o, None)

    slots.copy_(torch.randperm(9600)[:T])
    step(e, want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(c, out)
    for turn in range(4):
        x.copy_(torch.randn(x.shape))
        slots.copy_(torch.randint(0, 9600, (T,)))
        g.replay()
        torch.cuda.synchronize()
        step(e, want)
        assert torch.equal(out, want), turn


def test_the_binding_refuses():
    q = need_gpu()
    c = Cache(q, 2, 4, 2, 64, "int8", 64, True)
    x = torch.zeros((3, 2, 64), device="cuda")
    s = torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (lambda: q.kv_cache_write(x, None, s.int(), c.h, None),
                lambda: q.kv_cache_write(x, x, s, c.h, None),
                lambda: q.kv_cache_write(None, None, s, c.h, None),
                lambda: q.kv_cache_write(x[:2], None, s, c.h, None),
                lambda: q.kv_cache_write(x.transpose(1, 2), None, s, c.h, None),
                lambda: q.kv_cache_write(x.cpu(), None, s, c.h, None),
                lambda: q.kv_cache_read(c.h, None, s.cpu(), x, None),
                lambda: q.make_kv_cache(c.codes, c.scales, c.zeros[:, :, :1], 64, "int8", 64),
                lambda: q.make_kv_cache(c.codes, c.scales, c.zeros, 64, "e4m3", 64),
                lambda: q.make_kv_cache(c.codes, c.scales, None, 64, "int4", 64)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        q.kv_cache_write(x.half(), None, s, c.h, None)
