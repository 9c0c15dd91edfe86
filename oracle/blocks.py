"""Oracle of the operators on a paged cache with a scale per block of tokens and head, and of
drafted tokens (test infrastructure only).  fp64 throughout; what the operators hold in fp32 (scales,
the integer grid's quotients) is rounded to fp32 where they round it; the pages are whole numbers.

Sources: "LLM quantization principles: GPTQ, AWQ, GGUF", §2.1 (round(x / scale)); "AWQ, MinMax, GPTQ
calibration in Model Optimizer", §2 (scale = amax / qmax).  Parity unpinned by the pages: the block
of tokens, its growth by powers of two, the pages' order, the drafts' acceptance.
"""
from __future__ import annotations

import math

import numpy as np

from . import lowp
from .quantizer import f32


def values(codes: np.ndarray, fmt: str) -> np.ndarray:
    return lowp.e4m3_decode(codes) if fmt == "e4m3" else codes.astype(np.float64) - 128.0


def encode(x: np.ndarray, scale: np.ndarray, fmt: str) -> np.ndarray:
    with np.errstate(invalid="ignore"):
        q = x / scale
        if fmt == "e4m3":
            return lowp.e4m3_encode(q)
        q = np.rint(f32(q)) + 128.0
        return np.where(np.isnan(q), 0, np.clip(q, 0, 255)).astype(np.uint8)


def need_of(a: np.ndarray, fmt: str) -> np.ndarray:
    return np.maximum(f32(a / 448.0 if fmt == "e4m3" else 2.0 * a / 255.0), lowp.MIN_SCALE)


def write(codes, scales, fmt, x, table, lengths, starts):
    """codes [pages, page, heads, dim] (uint8) and scales [pages, blocks, heads] (fp64), in place;
    returns whether a row had no page."""
    pages, page = codes.shape[:2]
    B = page // scales.shape[1]
    bad = False
    for i, n in enumerate(lengths):
        s0, s1 = starts[i], starts[i + 1]
        rows = {n - (s1 - s0) + r: s0 + r for r in range(s1 - s0) if n - (s1 - s0) + r >= 0}
        for b0 in sorted({p - p % B for p in rows}):
            at = [p for p in range(b0, b0 + B) if p in rows]
            e = b0 // page
            pg = table[i][e] if e < len(table[i]) else -1
            if not 0 <= pg < pages:
                bad = True
                continue
            new = x[[rows[p] for p in at]]
            a = np.where(np.isfinite(new), np.abs(new), 0.0).max(axis=(0, 2))
            need = need_of(a, fmt)
            o, blk = b0 % page, (b0 % page) // B
            for h in range(codes.shape[2]):
                s = need[h] if a[h] > 0 else 1.0
                old = scales[pg, blk, h]
                if at[0] > b0 and np.isfinite(old) and old >= lowp.MIN_SCALE:
                    s = old
                    while a[h] > 0 and s < need[h]:
                        s *= 2.0
                    if s != old:
                        k = codes[pg, o:o + at[0] - b0, h]
                        v = values(k, fmt) * (old / s)
                        k[...] = lowp.e4m3_encode(v) if fmt == "e4m3" else (np.rint(v) + 128).astype(np.uint8)
                scales[pg, blk, h] = s
                for p, r in zip(at, new[:, h]):
                    codes[pg, p % page, h] = encode(r, s, fmt)
    return bad


def attention(q, kc, ks, vc, vs, fmt, table, lengths, starts, causal=True, window=0, scale=None):
    """(out, lse, mag, smax): mag = sum of w |v| and smax = the largest sum of |scale q k| of a row's
    keys, for error bounds.  Rows of no sequence are NaN."""
    T, HQ, D = q.shape
    pages, page, H = kc.shape[:3]
    B = page // ks.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.full((T, HQ, D), np.nan), np.full((T, HQ), np.nan)
    mag, smax = np.zeros((T, HQ, D)), np.zeros((T, HQ))
    for i, n in enumerate(lengths):
        s0, s1 = starts[i], starts[i + 1]
        pos = np.arange(n)
        e = pos // page
        pg = np.array([table[i][j] if j < len(table[i]) else -1 for j in e], dtype=np.int64)
        there = (pg >= 0) & (pg < pages)
        g, sl = np.where(there, pg, 0), pos % page
        for t in range(s0, s1):
            own = n - (s1 - s0) + t - s0
            see = there.copy()
            if causal:
                see &= pos <= own
                if window:
                    see &= pos > own - window
            for h in range(HQ):
                kh = h // (HQ // H)
                if not see.any():
                    out[t, h], lse[t, h] = 0.0, -np.inf
                    continue
                k = values(kc[g, sl, kh], fmt)[see] * ks[g, sl // B, kh][see, None]
                v = values(vc[g, sl, kh], fmt)[see] * vs[g, sl // B, kh][see, None]
                with np.errstate(invalid="ignore"):
                    s = k @ q[t, h] * scale
                    m = s.max()
                    w = np.exp(s - m)
                    out[t, h] = w @ v / w.sum()
                    lse[t, h] = m + np.log(w.sum())
                    mag[t, h] = w @ np.abs(v) / w.sum()
                    smax[t, h] = (np.abs(k) @ np.abs(q[t, h])).max() * scale
    return out, lse, mag, smax


def pages_of(n: int, page: int) -> int:
    return -(-max(n, 0) // page)


def fork(table, lengths, refs, parents, page):
    """(new_table, new_lengths, new_refs)"""
    refs, width = list(refs), len(table[0]) if len(table) else 0
    new_table, new_lengths = [], []
    for i, n in enumerate(lengths):
        for j in range(pages_of(n, page)):
            refs[table[i][j]] -= 1
    for p in parents:
        n = lengths[p] if p >= 0 else 0
        row = [table[p][j] if j < pages_of(n, page) else -1 for j in range(width)]
        for j in range(pages_of(n, page)):
            refs[row[j]] += 1
        new_table.append(row)
        new_lengths.append(n)
    return new_table, new_lengths, refs


def resize(table, lengths, refs, new_lengths, page):
    """(table, lengths, refs, src, dst, info) after the call."""
    table, lengths, refs = [list(r) for r in table], list(lengths), list(refs)
    R, width, info = len(table), len(table[0]), 0
    want = []
    for i, n in enumerate(new_lengths):
        if pages_of(n, page) > width:
            info |= 1
            n = -1
        want.append(lengths[i] if n < 0 else n)
    for i in range(R):
        if want[i] < lengths[i]:
            for j in range(pages_of(want[i], page), pages_of(lengths[i], page)):
                refs[table[i][j]] -= 1
                table[i][j] = -1
            lengths[i] = want[i]
    writers = {}
    for i in range(R):
        if want[i] > lengths[i] and lengths[i] % page:
            writers.setdefault(table[i][lengths[i] // page], []).append(i)
    copies = set()
    for pg, who in writers.items():
        if refs[pg] > 1:
            copies |= set(who[:-1] if len(who) == refs[pg] else who)
    src, dst = [-1] * R, [-1] * R
    free = [p for p, n in enumerate(refs) if n == 0]
    need = sum((i in copies) + max(pages_of(want[i], page) - pages_of(lengths[i], page), 0) for i in range(R))
    if need > len(free):
        return table, lengths, refs, src, dst, info | 2
    for i in range(R):
        if want[i] <= lengths[i]:
            continue
        o = pages_of(lengths[i], page)
        if i in copies:
            src[i], dst[i] = table[i][o - 1], free.pop(0)
            refs[src[i]] -= 1
            refs[dst[i]] = 1
            table[i][o - 1] = dst[i]
        for j in range(o, pages_of(want[i], page)):
            table[i][j] = free.pop(0)
            refs[table[i][j]] = 1
        lengths[i] = want[i]
    return table, lengths, refs, src, dst, info


def compact(table, refs):
    """(new_table, new_refs, src, dst, count)"""
    live = [p for p, n in enumerate(refs) if n > 0]
    L = len(live)
    src = [p for p in live if p >= L]
    dst = [p for p in range(L) if refs[p] <= 0]
    to = dict(zip(src, dst))
    new = [0] * len(refs)
    for p in live:
        new[to.get(p, p)] = refs[p]
    return [[to.get(p, p) for p in row] for row in table], new, src, dst, L


def softmax(x: np.ndarray, temperature: float) -> np.ndarray:
    """NaN throughout where x holds a NaN, +inf, or nothing but -inf."""
    x = np.asarray(x, dtype=np.float64)
    if temperature == 0:
        p = np.zeros_like(x)
        p[int(np.argmax(x))] = 1.0
        return p if np.isfinite(x.max()) else np.full_like(x, np.nan)
    with np.errstate(invalid="ignore"):
        e = np.exp((x - x.max()) / temperature)
        return e / e.sum()


def verify(target, draft, ids, starts, u, u_next, temperatures=None):
    """(accepted, tokens, logprobs, margin): margin = how near the closest decision was to going
    the other way, relative to the probabilities it compares."""
    *out, accepts, draws = verify_margins(target, draft, ids, starts, u, u_next, temperatures)
    return *out, min([m for m, _ in accepts] + [draws])


def verify_margins(target, draft, ids, starts, u, u_next, temperatures=None):
    """(accepted, tokens, logprobs, accepts, draws): accepts = for each acceptance or refusal by two
    numbers, |u q / p - 1| and how far the token's logits are below their rows' largest, in
    temperatures (the target's and the drafter's in all); draws = how near the closest draw came to its border."""
    T, V = target.shape
    S = len(starts) - 1
    accepted, tokens, logprobs = np.zeros(S, np.int64), np.full(T, -1, np.int64), np.zeros(T)
    accepts, draws = [], math.inf
    for i in range(S):
        temp = 1.0 if temperatures is None else float(temperatures[i])
        r, end = starts[i], starts[i + 1]
        while r < end:
            p = softmax(target[r], temp)
            w = p
            if r < end - 1:
                x = int(ids[r])
                q = None
                if 0 <= x < V:
                    if draft is None or temp == 0:
                        q = np.zeros(V)
                        q[x] = 1.0
                    else:
                        q = softmax(draft[r], temp)
                    good = p[x] == 1.0 if temp == 0 else u[r] * q[x] < p[x]
                    if temp != 0 and np.isfinite(p[x]) and np.isfinite(q[x]) and p[x] > 0:
                        below = (target[r].max() - target[r][x]) / temp
                        if draft is not None:
                            below += (draft[r].max() - draft[r][x]) / temp
                        accepts.append((abs(u[r] * q[x] / p[x] - 1.0), below))
                    if good:
                        tokens[r], logprobs[r] = x, 0.0 if temp == 0 else math.log(p[x])
                        accepted[i] += 1
                        r += 1
                        continue
                elif draft is not None and temp != 0:
                    q = softmax(draft[r], temp)
                if q is not None:
                    w = np.nan_to_num(np.maximum(p - q, 0.0), nan=0.0)
                    w = w if w.sum() > 0 else p
            if np.isnan(p).any():
                break
            c = np.cumsum(w)
            border = u_next[i] * c[-1]
            v = int(np.searchsorted(c, border, side="right"))
            if temp != 0:
                draws = min(draws, np.abs(c[:-1][w[:-1] > 0] - border).min(initial=np.inf) / c[-1])
            tokens[r], logprobs[r] = v, 0.0 if temp == 0 else math.log(p[v])
            break
    return accepted, tokens, logprobs, accepts, draws
