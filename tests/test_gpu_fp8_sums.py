"""GPU: the e4m3 products' sums beside outliers, on every tile.

An activation channel far above its neighbours is what the block scales are for: its
products must not cost the neighbours' their digits.  Two outlier channels of a block
that cancel leave integer sums below 2^24, so every fp32 sum is exact, in any order,
and Y is compared for equality; over inexact data the bound is fp32's alone, whatever
the type of Y (with A = sum |x w|: a block's products are added in fp32, 127 additions
off by at most a whole step each, two roundings of the scales, nb fmas:
(127 * 2 + 2 + nb) 2^-24 A, then half a step of Y's type)."""
import numpy as np
import pytest

from oracle import lowp

from gpu_util import host, need_gpu, say, torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U8 = torch.uint8

# decode kernels, narrow and wide tiles, with splits and without
SIZES = [(1, 300, 272), (16, 8200, 144), (32, 100, 400), (33, 300, 2064), (100, 1000, 4112),
         (300, 520, 272), (512, 1100, 2064), (300, 11010, 272), (2600, 4100, 272), (2050, 7700, 144)]


def _outliers(rng, T, m, n):
    """Codes of integers: -3 .. 3, and in each block two columns, anywhere, where X holds
    448 and the rows of W +448 and -448 (or 0)."""
    x, w = rng.integers(-3, 4, size=(T, n)), rng.integers(-3, 4, size=(m, n))
    for b0 in range(0, n, 128):
        size = min(128, n - b0)
        p, q = b0 + rng.choice(size, 2, replace=False)
        x[:, [p, q]] = 448
        w[:, p] = rng.choice([-448, 0, 448], size=m)
        w[:, q] = -w[:, p]
    codes = [torch.from_numpy(lowp.e4m3_encode(v.astype(float))).cuda() for v in (x, w)]
    return codes[0], codes[1], torch.from_numpy(x).float().cuda(), torch.from_numpy(w).float().cuda()


@pytest.mark.parametrize("ydt", [F32, BF])
@pytest.mark.parametrize("T,m,n", SIZES)
def test_cancelling_outliers_leave_the_rest(T, m, n, ydt):
    q = need_gpu()
    rng = np.random.default_rng(T + m + n)
    xc, wc, x, w = _outliers(rng, T, m, n)
    xs, ws = torch.ones((-(-n // 128), T), device="cuda"), torch.ones((-(-m // 128), -(-n // 128)), device="cuda")
    Y = torch.full((T, m), 7.0, dtype=ydt, device="cuda")
    say("fp8 product beside outliers", T, m, n, ydt)
    q.fp8_gemm(xc, xs, wc, ws, Y)
    # the outliers' products leave nothing: the sums without them (in fp32, exact)
    big = (x == 448).any(0)
    x[:, big] = 0
    assert torch.equal(Y, (x @ w.T).to(ydt))


@pytest.mark.parametrize("ydt", [F32, BF])
@pytest.mark.parametrize("T,m,n", [(5, 300, 1040), (40, 260, 1040), (300, 520, 2064), (300, 4200, 400)])
def test_outlier_channels_within_fp32s_bound(T, m, n, ydt):
    q = need_gpu()
    rng = np.random.default_rng(T * 31 + m + n)
    xv = rng.standard_t(4, size=(T, n))
    xv[:, rng.choice(n, 6, replace=False)] *= 1000.0
    xc, xs = lowp.quantize_rows(xv)
    wc, ws = lowp.quantize_blocks(rng.normal(size=(m, n)) * 0.02)
    ref, mag = lowp.gemm(xc, xs, wc, ws)
    Y = torch.empty((T, m), dtype=ydt, device="cuda")
    say("fp8 product, outlier channels", T, m, n, ydt)
    q.fp8_gemm(torch.from_numpy(xc).cuda(), torch.from_numpy(xs).float().cuda(), torch.from_numpy(wc).cuda(),
               torch.from_numpy(ws).float().cuda(), Y)
    half = torch.finfo(ydt).eps / 2
    bound = (127 * 2 + 2 + xs.shape[0]) * 2.0 ** -24 * mag
    assert np.all(np.abs(host(Y.double()) - ref) <= bound * (1 + half) + half * np.abs(ref))


@pytest.mark.parametrize("T,m,n", [(40, 300, 272), (257, 8300, 272), (300, 8320, 400)])
def test_gated_product_beside_outliers(T, m, n):
    """g and u are integers / 64, exact in fp32; half a step of bf16 apart from that.  h
    is then off by 2^-20 (the exp, the sum, the quotient and the product), its codes by
    half a step (2^-4 relative, or half the smallest step 2^-9 times the scale)."""
    q = need_gpu()
    rng = np.random.default_rng(T + m)
    xc, gc, x, g = _outliers(rng, T, m, n)
    uc, u = gc.flip(0).contiguous(), g.flip(0)  # (the same columns hold the outliers)
    nb, mb = -(-n // 128), -(-m // 128)
    xs, ws = torch.full((nb, T), 1 / 64, device="cuda"), torch.ones((mb, nb), device="cuda")
    codes = torch.full((T, m), 0x55, dtype=U8, device="cuda")
    scales = torch.full((mb, T), -1.0, device="cuda")
    say("fp8 gated product beside outliers", T, m, n)
    q.fp8_gated_gemm(xc, xs, gc, ws, uc, ws, codes, scales)
    x[:, (x == 448).any(0)] = 0
    g, u = (((x @ v.T) / 64).to(BF).double().cpu().numpy() for v in (g, u))
    h = g / (1 + np.exp(-g)) * u
    s = host(scales).astype(np.float64)
    for b in range(mb):
        want = np.abs(h[:, b * 128:(b + 1) * 128]).max(1) / 448
        assert np.all(np.abs(s[b] - want) <= 2.0 ** -19 * want), b
    sp = np.repeat(s, 128, 0)[:m].T
    back = lowp.e4m3_decode(host(codes)) * sp
    assert np.all(np.abs(back - h) <= np.abs(h) * (2.0 ** -4 + 2.0 ** -19) + 2.0 ** -10 * sp)
