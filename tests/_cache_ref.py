"""Plain 64-bit reference of the paged 8-bit KV cache (numpy), for the parity tests."""
from __future__ import annotations

import numpy as np

QMAX = {"e4m3": 448.0, "int8": 127.0}
TINY = 2.0 ** -96


def code_values(fmt: str) -> np.ndarray:
    """Value of each of the 256 code bytes (two e4m3 bytes are NaN)."""
    b = np.arange(256)
    if fmt == "int8":
        return np.where(b < 128, b, b - 256).astype(np.float64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e.astype(np.float64) - 10))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


def to_codes(x: np.ndarray, fmt: str) -> np.ndarray:
    """Code values nearest to x (ties to even, clamped); NaN stays NaN in e4m3, 0 in int8."""
    if fmt == "int8":
        return np.clip(np.nan_to_num(np.rint(x), nan=0.0, posinf=127, neginf=-127), -127, 127)
    with np.errstate(invalid="ignore"):
        e = np.floor(np.log2(np.maximum(np.minimum(np.abs(x), 1e30), 2.0 ** -6)))
        step = np.exp2(e - 3)
        return np.clip(np.rint(x / step) * step, -448, 448)


def scale_of(big: np.ndarray, fmt: str) -> np.ndarray:
    """Least number of 8 significant bits that is >= max(2^-96, big) / qmax."""
    s = np.maximum(big, TINY) / QMAX[fmt]
    unit = np.exp2(np.floor(np.log2(s)) - 7)
    return np.ceil(s / unit) * unit


def tables(ps, P, max_len, add, lens, tab, ring, state, max_tokens):
    """The next step's tables; returns a dict of copies (the inputs stay as they are)."""
    B = len(add)
    lens, tab, ring = lens.copy(), tab.copy(), ring.copy()
    head, count = int(state[0]), int(state[1])
    pages = lambda n: -(-n // ps)  # noqa: E731
    status, need, back, new = 0, 0, 0, 0
    for s in range(B):
        if not 0 <= lens[s] <= max_len:
            status |= 8
        elif add[s] < 0:
            back += pages(int(lens[s]))
        elif int(lens[s]) + int(add[s]) > max_len:
            status |= 2
        else:
            need += pages(int(lens[s]) + int(add[s])) - pages(int(lens[s]))
            new += int(add[s])
    if not (0 <= head < P and 0 <= count <= P):
        status |= 8
    elif need > count:
        status |= 1
    elif count - need + back > P:
        status |= 8
    if new > max_tokens:
        status |= 4
    cu, slots = np.zeros(B + 1, np.int32), np.full(max_tokens, -1, np.int32)
    if status:
        return dict(lens=lens, tables=tab, ring=ring, state=np.array([head, count]), cu=cu, slots=slots, status=status)
    taken, given = 0, 0
    for s in range(B):
        n, h = max(int(add[s]), 0), pages(int(lens[s]))
        cu[s + 1] = cu[s] + n
        if add[s] < 0:
            for j in range(h):
                ring[(head + count + given) % P] = tab[s, j]
                given += 1
            lens[s] = 0
            continue
        for j in range(h, pages(int(lens[s]) + n)):
            tab[s, j] = ring[(head + taken) % P]
            taken += 1
        for j in range(n):
            pos = int(lens[s]) + j
            page = tab[s, pos // ps]
            slots[cu[s] + j] = page * ps + pos % ps if 0 <= page < P else -1
        lens[s] += n
    return dict(lens=lens, tables=tab, ring=ring, state=np.array([(head + taken) % P, count - taken + given]), cu=cu,
                slots=slots, status=0)


def append(fmt, ps, bs, x, cu, lens, slots, codes, scales):
    """New rows x [n, H, D] (float64) into copies of codes [P, H, ps, D] (values) and scales."""
    codes, scales = codes.copy(), scales.copy()
    for s in range(len(lens)):
        n = cu[s + 1] - cu[s]
        pos, t = lens[s] - n, cu[s]
        while pos < lens[s]:
            off = pos % ps
            m = min(ps - off, lens[s] - pos)
            if slots[t] >= 0:
                page = slots[t] // ps
                rows = x[t:t + m].transpose(1, 0, 2)
                sc = scale_of(np.where(np.isfinite(rows), np.abs(rows), 0).max((1, 2)), fmt)
                if off:
                    new = np.maximum(sc, scales[page])
                    grew = new > scales[page]
                    moved = to_codes(codes[page, :, :off] * scales[page][:, None, None] / new[:, None, None], fmt)
                    codes[page, :, :off] = np.where(grew[:, None, None], moved, codes[page, :, :off])
                    sc = new
                codes[page, :, off:off + m] = to_codes(rows / sc[:, None, None], fmt)
                scales[page] = sc
            pos, t = pos + m, t + m
    return codes, scales


def pooled(ps, bs, cu, lens, tab, codes, scales):
    """{(s, b): (mean, mean of magnitudes)} of the blocks that the step completes, [H, D] each."""
    out = {}
    for s in range(len(lens)):
        for b in range((lens[s] - (cu[s + 1] - cu[s])) // bs, lens[s] // bs):
            pages = tab[s, b * bs // ps:(b + 1) * bs // ps]
            v = codes[pages] * scales[pages][:, :, None, None]
            out[s, b] = v.sum((0, 2)) / bs, np.abs(v).sum((0, 2)) / bs
    return out


def decode(q, kc, vc, ks, vs, kbar, lens, tab, ps, bs, k, scale):
    """q [B, Hq, D] float64; codes as values.  Returns O, LSE, sel, and what the error bounds need:
    wide = sum_j p_j |v_j| and zabs = max_j scale * sum_d |q_d k_jd|."""
    B, Hq, D = q.shape
    G, P = Hq // kc.shape[1], kc.shape[0]
    O, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    sel, wide, zabs = np.full((B, Hq, k), -1, np.int64), np.zeros((B, Hq, D)), np.zeros((B, Hq))
    for s in range(B):
        n = int(lens[s])
        if n == 0:
            continue
        i = (n - 1) // bs
        for h in range(Hq):
            blocks = [i]
            if i and k > 1:
                score = kbar[s, :i, h // G] @ q[s, h]
                score = np.where(np.isnan(score), -np.inf, score)
                blocks += list(np.argsort(-score, kind="stable")[:k - 1])
            sel[s, h, :len(blocks)] = blocks
            pos = np.concatenate([np.arange(b * bs, min((b + 1) * bs, n)) for b in blocks])
            page = tab[s, pos // ps]
            ok = (page >= 0) & (page < P)
            pos, page = pos[ok], page[ok]
            if not pos.size:
                continue
            key = kc[page, h // G, pos % ps] * ks[page, h // G, None]
            val = vc[page, h // G, pos % ps] * vs[page, h // G, None]
            z = key @ q[s, h] * scale
            zabs[s, h] = (np.abs(key) @ np.abs(q[s, h])).max() * scale
            top = z.max()
            p = np.exp(z - top)
            lse[s, h] = top + np.log(p.sum())
            p /= p.sum()
            O[s, h], wide[s, h] = p @ val, p @ np.abs(val)
    return O, lse, sel, wide, zabs
