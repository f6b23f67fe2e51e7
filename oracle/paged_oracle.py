"""Plain fp64 oracle of the paged key/value cache (test infrastructure only).

Codes, scales and attention from their definitions, with numpy in 64 bits:
rows are quantised by comparing the exact quotient with every border, caches
are plain arrays addressed through the page table one token at a time.
"""

from __future__ import annotations

import numpy as np

QMAX = {"int8": 127.0, "e4m3": 448.0}


def e4m3_value(byte):
    """Value of an e4m3 code (bias 7, subnormals below 2^-6, 0x7f / 0xff NaN)."""
    b = np.asarray(byte).astype(np.int64)
    s, e, m = np.where(b & 128, -1.0, 1.0), (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(np.float64) - 10))
    return np.where((b & 127) == 127, np.nan, s * v)


_E4M3_GRID = e4m3_value(np.arange(127))  # the non-negative values, ascending


def code_value(codes, kind):
    return e4m3_value(codes) if kind == "e4m3" else np.asarray(codes).astype(np.float64)


def quantise(x, kind):
    """Codes (int8, or uint8 bits of e4m3) and float32 scales of rows x [..., D] (float64 holding fp32 or bf16 values).

    x * M / a in fp64: x * M is exact (24 + 9 bits) and the quotient of two such
    numbers differs from a border (8 bits) by more than fp64's rounding unless it
    lies on it, where the division is exact."""
    x = np.asarray(x, np.float64)
    M = QMAX[kind]
    a = np.max(np.abs(x), axis=-1, keepdims=True)
    bad = ~np.isfinite(x).all(axis=-1, keepdims=True)
    zero = (a == 0) & ~bad
    with np.errstate(all="ignore"):
        t = np.where(bad | zero, 0.0, np.abs(x) * M / np.where(bad | zero, 1.0, a))
        scale = np.where(bad, np.nan, np.where(zero, 0.0, a)).astype(np.float32) / np.float32(M)
    sign = np.signbit(x) & ~bad
    if kind == "int8":
        c = np.rint(t)
        codes = np.where(sign, -c, c).astype(np.int8)
    else:
        i = np.clip(np.searchsorted(_E4M3_GRID, t, side="right") - 1, 0, 125)
        lo, hi = _E4M3_GRID[i], _E4M3_GRID[i + 1]
        up = (t - lo > hi - t) | ((t - lo == hi - t) & (i % 2 == 1))
        codes = ((i + up) | np.where(sign, 128, 0)).astype(np.uint8)
    return codes, scale[..., 0]


def places(token_start, seq_len, table, page_size):
    """(packed row, sequence, position, page, slot) of every new token."""
    for s in range(len(seq_len)):
        n = int(token_start[s + 1]) - int(token_start[s])
        for i in range(n):
            pos = int(seq_len[s]) - n + i
            yield int(token_start[s]) + i, s, pos, int(table[s, pos // page_size]), pos % page_size


def attend(q, k_pages, v_pages, table, seq_len, token_start, scale, out, bounds=None):
    """out[t, h] (fp64, given) overwritten for the tokens of sequences; pages [n, Hkv, page, D] are values in fp64.

    bounds: a dict that receives, in out's shape, what error bounds need:
    "A" sum_j w_j |v_j| and "B" sum_j w_j s_j (|v_j| + |out|) with s_j = scale sum_d |q_d k_jd|."""
    _, Hkv, ps, D = k_pages.shape
    G = q.shape[1] // Hkv
    if bounds is not None:
        bounds["A"], bounds["B"] = np.zeros_like(out), np.zeros_like(out)
    for s in range(len(seq_len)):
        a, b, n = int(token_start[s]), int(token_start[s + 1]), int(seq_len[s])
        if a == b:
            continue
        pages = table[s, :-(-n // ps)]
        k = k_pages[pages].transpose(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n]
        v = v_pages[pages].transpose(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n]
        sees = np.arange(n)[None, :] <= (n - (b - a) + np.arange(b - a))[:, None]
        for h in range(q.shape[1]):
            kh, vh, qh = k[h // G], v[h // G], q[a:b, h]
            z = np.where(sees, scale * (qh @ kh.T), -np.inf)
            w = np.exp(z - z.max(axis=1, keepdims=True))
            w /= w.sum(axis=1, keepdims=True)
            o = w @ vh
            out[a:b, h] = o
            if bounds is not None:
                ws = w * (scale * (np.abs(qh) @ np.abs(kh).T))
                bounds["A"][a:b, h] = w @ np.abs(vh)
                bounds["B"][a:b, h] = ws @ np.abs(vh) + ws.sum(axis=1, keepdims=True) * np.abs(o)
    return out
