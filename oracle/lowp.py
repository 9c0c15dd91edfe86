"""Oracle of the low-precision operators (test infrastructure only): e4m3 with
block scales and its product, the quantized key/value cache, token log
probabilities.  fp64 throughout; what the operators hold in fp32 (scales, the
integer grid's quotients) is rounded to fp32 where they round it.

Sources: "AWQ, MinMax, GPTQ calibration in Model Optimizer", §2 (scale = amax /
qmax); "LLM quantization principles: GPTQ, AWQ, GGUF", §2.1 (the affine grid);
"Quantized deployment, 1.5 TB to 250 GB", §3.1 (perplexity).  Parity unpinned by
the pages: the block of 128, the smallest scale 2^-126, the cache's layout.
"""
from __future__ import annotations

from typing import Optional, Tuple

import numpy as np

from . import quantizer
from .quantizer import f32

BLOCK = 128
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126


def e4m3_table() -> np.ndarray:
    """Value of each of the 256 codes (sign, 4 exponent bits with bias 7, 3
    mantissa bits; no infinities, 0x7F and 0xFF are NaN)."""
    code = np.arange(256)
    e, m = (code >> 3) & 15, code & 7
    mag = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    mag = np.where((code & 127) == 127, np.nan, mag)
    return np.where(code >= 128, -mag, mag)


_TABLE = e4m3_table()
_MAG = _TABLE[:127]


def e4m3_encode(v: np.ndarray) -> np.ndarray:
    """Code of the nearest e4m3 value, ties to the even code, +-448 at most;
    non-finite values give the NaN code.  The sign of v is kept."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isfinite(v), v, 0.0)), E4M3_MAX)
    hi = np.clip(np.searchsorted(_MAG, a), 1, 126)  # _MAG[hi - 1] < a <= _MAG[hi]
    dl, dh = a - _MAG[hi - 1], _MAG[hi] - a
    code = np.where(dl < dh, hi - 1, np.where(dl > dh, hi, hi - hi % 2))
    code = np.where(np.isfinite(v), code, 127)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def e4m3_decode(code: np.ndarray) -> np.ndarray:
    return _TABLE[np.asarray(code, dtype=np.uint8)]


def e4m3_scale(amax: np.ndarray) -> np.ndarray:
    amax = np.asarray(amax, dtype=np.float64)
    return np.where(amax == 0, 1.0, np.maximum(f32(amax / E4M3_MAX), MIN_SCALE))


def _amax(v: np.ndarray, axis) -> np.ndarray:
    return np.where(np.isfinite(v), np.abs(v), 0.0).max(axis=axis)


def quantize_rows(x: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """codes [T, n], scales [ceil(n / 128), T]."""
    x = np.asarray(x, dtype=np.float64)
    T, n = x.shape
    codes = np.empty((T, n), np.uint8)
    scales = np.empty((-(-n // BLOCK), T))
    for b in range(scales.shape[0]):
        c = slice(b * BLOCK, min(n, (b + 1) * BLOCK))
        scales[b] = e4m3_scale(_amax(x[:, c], 1))
        codes[:, c] = e4m3_encode(x[:, c] / scales[b][:, None])
    return codes, scales


def quantize_blocks(w: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """codes [m, n], scales [ceil(m / 128), ceil(n / 128)]."""
    w = np.asarray(w, dtype=np.float64)
    m, n = w.shape
    codes = np.empty((m, n), np.uint8)
    scales = np.empty((-(-m // BLOCK), -(-n // BLOCK)))
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = np.s_[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
            scales[i, j] = e4m3_scale(_amax(w[at], None))
            codes[at] = e4m3_encode(w[at] / scales[i, j])
    return codes, scales


def gemm(xc, xs, wc, ws) -> Tuple[np.ndarray, np.ndarray]:
    """Y [T, m] and, for error bounds, the sum of the products' magnitudes."""
    n = xc.shape[1]
    x = e4m3_decode(xc) * np.repeat(np.asarray(xs, np.float64), BLOCK, 0)[:n].T
    w = e4m3_decode(wc) * np.repeat(np.repeat(np.asarray(ws, np.float64), BLOCK, 0)[:wc.shape[0]],
                                    BLOCK, 1)[:, :n]
    return x @ w.T, np.abs(x) @ np.abs(w).T


def kv_quantize(x: np.ndarray, fmt: str, group: int, asym: bool):
    """x [rows, dim] -> codes [rows, dim] (not packed), scales and zeros [rows, groups]."""
    x = np.asarray(x, dtype=np.float64)
    rows, dim = x.shape
    group = dim if group <= 0 else min(group, dim)
    ng = -(-dim // group)
    codes = np.empty((rows, dim), np.uint8)
    scales, zeros = np.empty((rows, ng)), np.zeros((rows, ng))
    for j in range(ng):
        c = slice(j * group, min(dim, (j + 1) * group))
        if fmt == "e4m3":
            scales[:, j] = e4m3_scale(_amax(x[:, c], 1))
            codes[:, c] = e4m3_encode(x[:, c] / scales[:, j, None])
        else:
            bits = 4 if fmt == "int4" else 8
            scales[:, j], zeros[:, j] = quantizer.group_params(x[:, c], bits, sym=not asym)
            codes[:, c] = quantizer.quantize_codes(x[:, c], scales[:, j, None], zeros[:, j, None],
                                                   bits)
    return codes, scales, zeros


def kv_dequantize(codes, scales, zeros, fmt: str, group: int) -> np.ndarray:
    dim = codes.shape[1]
    group = dim if group <= 0 else min(group, dim)
    at = np.arange(dim) // group
    if fmt == "e4m3":
        return e4m3_decode(codes) * scales[:, at]
    return (codes.astype(np.float64) - zeros[:, at]) * scales[:, at]


def kv_pack(codes: np.ndarray, fmt: str) -> np.ndarray:
    return codes[..., 0::2] | codes[..., 1::2] << 4 if fmt == "int4" else codes


def logprobs(x: np.ndarray, ids: Optional[np.ndarray], top: int):
    """(logprob, entropy, top_ids, top_logprobs) of rows of logits, in fp64."""
    x = np.asarray(x, dtype=np.float64)
    T, V = x.shape
    lp, ent = np.zeros(T), np.zeros(T)
    tid, tlp = np.zeros((T, top), np.int64), np.zeros((T, top))
    for t in range(T):
        row = x[t]
        order = np.lexsort((np.arange(V), -np.where(np.isnan(row), -np.inf, row)))[:top]
        if np.isnan(row).any() or np.isposinf(row).any():
            logp, ent[t] = np.full(V, np.nan), np.nan
        elif np.isneginf(row).all():
            logp, ent[t] = row.copy(), 0.0
        else:
            m = row.max()
            logp = row - m - np.log(np.sum(np.exp(row - m)))
            p = np.exp(logp)
            ent[t] = -np.sum(p[p > 0] * logp[p > 0])
        tid[t], tlp[t] = order, logp[order]
        if ids is not None:
            i = int(ids[t])
            lp[t] = 0.0 if i < 0 else np.nan if i >= V else logp[i]
    return lp, ent, tid, tlp
