"""CPU: the low-precision oracle against closed forms, the format's own
definition and brute force."""
import numpy as np
import pytest

from oracle import lowp

torch = pytest.importorskip("torch")


def test_e4m3_table_is_the_format():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(t, nan=-1.0), np.nan_to_num(lowp.e4m3_table(), nan=-1.0))
    assert np.isnan(t[127]) and np.isnan(t[255]) and t[126] == 448.0 and t[1] == 2.0 ** -9


def test_e4m3_encode_is_nearest_with_ties_to_even():
    table = lowp.e4m3_table()[:127]
    # every value, every border and its two neighbours
    border = (table[1:] + table[:-1]) / 2
    v = np.concatenate([table, border, np.nextafter(border, 0), np.nextafter(border, 1e9)])
    code = lowp.e4m3_encode(v)
    brute = np.abs(v[:, None] - table[None]).argmin(1)  # lowest code of a tie
    tie = np.isin(v, border)
    brute = np.where(tie & (brute % 2 == 1), brute + 1, brute)
    assert np.array_equal(code, brute)
    assert np.array_equal(lowp.e4m3_encode(-v[1:]), brute[1:] + 128)
    assert lowp.e4m3_encode(np.array([460.0]))[0] == 126
    assert list(lowp.e4m3_encode(np.array([np.nan, np.inf, -np.inf]))) == [127, 127, 255]


def test_scales_and_blocks():
    assert lowp.e4m3_scale(0.0) == 1.0
    assert lowp.e4m3_scale(448.0) == 1.0
    assert lowp.e4m3_scale(1e-44) == 2.0 ** -126
    rng = np.random.default_rng(0)
    w = rng.normal(size=(130, 140))
    c, s = lowp.quantize_blocks(w)
    assert s.shape == (2, 2)
    back = lowp.e4m3_decode(c) * np.repeat(np.repeat(s, 128, 0)[:130], 128, 1)[:, :140]
    # half a step of 3 mantissa bits, and half the smallest step under a block's normals
    assert np.all(np.abs(back - w) <= np.maximum(np.abs(w) * 2.0 ** -4, 2.0 ** -10 * s.max()))
    x = w.T[:5]
    cr, sr = lowp.quantize_rows(x)
    assert sr.shape == (2, 5) and np.array_equal(cr[0, 128:], lowp.e4m3_encode(x[0, 128:] / sr[1, 0]))


def test_gemm_is_the_dequantized_product():
    rng = np.random.default_rng(1)
    xc, xs = lowp.quantize_rows(rng.normal(size=(3, 272)))
    wc, ws = lowp.quantize_blocks(rng.normal(size=(150, 272)))
    y, _ = lowp.gemm(xc, xs, wc, ws)
    t, r = 2, 140
    want = sum(xs[k // 128, t] * ws[r // 128, k // 128] * lowp.e4m3_decode(xc[t, k])
               * lowp.e4m3_decode(wc[r, k]) for k in range(272))
    assert abs(y[t, r] - want) <= 1e-12 * abs(want)


@pytest.mark.parametrize("fmt,asym", [("int4", True), ("int8", True), ("int4", False), ("e4m3", False)])
def test_cache_rows_come_back_within_half_a_step(fmt, asym):
    rng = np.random.default_rng(2)
    x = rng.normal(size=(6, 80)).astype(np.float32).astype(np.float64)
    c, s, z = lowp.kv_quantize(x, fmt, 32, asym)
    assert s.shape == (6, 3)
    back = lowp.kv_dequantize(c, s, z, fmt, 32)
    step = s[:, np.arange(80) // 32] * (1.0 if fmt != "e4m3" else np.maximum(
        2.0 ** -9, 2.0 ** -3 * np.abs(x / s[:, np.arange(80) // 32])))
    # asymmetric: the zero-point's rounding may push an end one step past the clamp
    assert np.all(np.abs(back - x) <= (1.01 if fmt != "e4m3" else 0.5) * step)
    packed = lowp.kv_pack(c, fmt)
    assert packed.shape[1] == (40 if fmt == "int4" else 80)


def test_logprobs_against_softmax_and_edge_rows():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(6, 11)) * 3
    x[1] = -np.inf
    x[2, 3] = np.nan
    x[3, 4] = np.inf
    x[4, 5:] = -np.inf
    x[5] = 1.0
    lp, ent, tid, tlp = lowp.logprobs(x, np.array([2, 0, 1, 1, 2, -1]), 4)
    p = np.exp(x[0]) / np.exp(x[0]).sum()
    assert abs(lp[0] - np.log(p[2])) < 1e-12 and abs(ent[0] + (p * np.log(p)).sum()) < 1e-12
    assert lp[1] == -np.inf and ent[1] == 0 and list(tid[1]) == [0, 1, 2, 3]
    assert np.isnan(lp[2]) and np.isnan(ent[2]) and np.isnan(lp[3]) and 3 not in tid[2]
    assert abs(ent[5] - np.log(11)) < 1e-12 and lp[5] == 0 and list(tid[5]) == [0, 1, 2, 3]
