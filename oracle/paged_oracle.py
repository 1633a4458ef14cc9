"""fp64 CPU oracle of the paged-cache operators: a plain loop over sequences, pages, heads and rows.

Shares no code with the library.  The cache is held as the values its elements stand for, e4m3 pages as (value in units
of the scale, scale)."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """Round to nearest even on the e4m3 grid (steps 2^-9 below 2^-6, else 2^(exponent - 3)); not finite -> NaN."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        ex = np.floor(np.log2(np.maximum(np.abs(x), 1e-300)))
        step = np.exp2(np.maximum(ex, -6.0) - 3.0)
        y = np.rint(x / step) * step          # rint: ties to even multiples of the step
        y = np.clip(y, -E4M3_MAX, E4M3_MAX)
    return np.where(np.isfinite(x), y, np.nan)


def bf16_round(x: np.ndarray) -> np.ndarray:
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        ex = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126)))
        step = np.exp2(ex - 7.0)
        y = np.rint(x / step) * step
    return np.where(np.isfinite(x), y, x)


def pow2_scale(amax: float) -> float:
    """Smallest power of two s with amax <= 448 s, in [2^-64, 2^119]; 1 for 0."""
    if amax == 0.0:
        return 1.0
    e = -64
    while e < 119 and amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def rotate(x: np.ndarray, cos_sin_row: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [H, D]: the first len(cos_sin_row) elements of each head rotated, in fp32 with every operation rounded."""
    y = np.array(x, np.float32)
    rot = cos_sin_row.shape[0]
    half = rot // 2
    for i in range(half):
        a_at, b_at = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        c, s = np.float32(cos_sin_row[i]), np.float32(cos_sin_row[half + i])
        a, b = np.float32(x[:, a_at]), np.float32(x[:, b_at])
        y[:, a_at] = a * c - b * s
        y[:, b_at] = b * c + a * s
    return y.astype(np.float64)


def append(cache: dict, table, kv_len, row_start, k, v, cos_sin=None, interleaved=False, pos=None, q=None):
    """cache: {"k", "v": [n_pages, Hkv, P, D] float64, "k_scale", "v_scale": [n_pages, Hkv] or None}, changed in place.
    Returns the rotated q rows (NaN where a row is padding)."""
    P = cache["k"].shape[2]
    q_out = None if q is None else np.full(q.shape, np.nan)
    for b in range(len(kv_len)):
        r0, r1 = int(row_start[b]), int(row_start[b + 1])
        n, kv = r1 - r0, int(kv_len[b])
        by_page: dict[int, list] = {}
        for j in range(n):
            p = kv - n + j
            rp = p if pos is None else int(pos[r0 + j])
            kr = np.asarray(k[r0 + j], np.float64)
            if cos_sin is not None:
                kr = rotate(kr, cos_sin[rp], interleaved)
            if q is not None:
                qr = np.asarray(q[r0 + j], np.float64)
                q_out[r0 + j] = bf16_round(rotate(qr, cos_sin[rp], interleaved)) if cos_sin is not None else qr
            by_page.setdefault(p // P, []).append((p % P, kr, np.asarray(v[r0 + j], np.float64)))
        for page, rows in by_page.items():
            pid = int(table[b][page])
            for name, at in (("k", 1), ("v", 2)):
                c, sc = cache[name], cache[name + "_scale"]
                if sc is None:
                    for row in rows:
                        c[pid, :, row[0]] = bf16_round(row[at])
                    continue
                first = rows[0][0]
                for h in range(c.shape[1]):
                    vals = np.array([row[at][h] for row in rows])
                    fin = np.abs(vals[np.isfinite(vals)])
                    amax = float(fin.max()) if fin.size else 0.0
                    new = pow2_scale(amax)
                    if first > 0:
                        old = float(sc[pid, h])
                        new = max(new, old) if amax > 0 else old
                        if new > old:
                            c[pid, h, :first] = e4m3_round(c[pid, h, :first] * (old / new))
                    sc[pid, h] = new
                    for row in rows:
                        c[pid, h, row[0]] = e4m3_round(row[at][h] / new)
    return q_out


def attention(cache: dict, table, kv_len, row_start, q, window=0, scale=None):
    """q [rows, Hq, D] -> o, lse and, for tolerances, per (row, head): the weighted mean of |v| and the largest
    sum over d of |q_d k_d| and of |k_d| among the visible keys."""
    P, hkv = cache["k"].shape[2], cache["k"].shape[1]
    rows, hq, D = q.shape
    G = hq // hkv
    scale = 1.0 / np.sqrt(D) if not scale else scale
    o = np.full((rows, hq, D), np.nan)
    lse, qk, kk = (np.full((rows, hq), np.nan) for _ in range(3))
    mean_abs = np.full((rows, hq, D), np.nan)
    for b in range(len(kv_len)):
        r0, r1 = int(row_start[b]), int(row_start[b + 1])
        n, kv = r1 - r0, int(kv_len[b])
        for h in range(hq):
            kv_head = h // G
            K, V = np.zeros((kv, D)), np.zeros((kv, D))
            for p in range(kv):
                pid = int(table[b][p // P])
                ks = 1.0 if cache["k_scale"] is None else float(cache["k_scale"][pid, kv_head])
                vs = 1.0 if cache["v_scale"] is None else float(cache["v_scale"][pid, kv_head])
                K[p], V[p] = cache["k"][pid, kv_head, p % P] * ks, cache["v"][pid, kv_head, p % P] * vs
            for j in range(n):
                at = kv - n + j
                keys = [p for p in range(kv) if p <= at and (not window or p > at - window)]
                r = r0 + j
                if not keys:
                    o[r, h], lse[r, h], mean_abs[r, h], qk[r, h], kk[r, h] = 0.0, -np.inf, 0.0, 0.0, 0.0
                    continue
                x = K[keys] @ q[r, h] * scale
                m = x.max()
                w = np.exp(x - m)
                o[r, h], lse[r, h] = w @ V[keys] / w.sum(), m + np.log(w.sum())
                mean_abs[r, h] = w @ np.abs(V[keys]) / w.sum()
                qk[r, h] = (np.abs(K[keys]) @ np.abs(q[r, h])).max() * scale
                kk[r, h] = np.abs(K[keys]).sum(1).max() * scale
    return o, lse, mean_abs, qk, kk
