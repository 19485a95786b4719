"""Routing of tokens to experts, 8-bit quantisation and products of 8-bit
weights with a scale for each block of 128 x 128, in float64 from the exact
inputs (the formulas of include/w4a16.h)."""
from __future__ import annotations

import numpy as np


# -------------------------------------------------------------- routing ---

def scores_ref(logits, score: str):
    """[M, E] float64 scores; NaN logits count as -infinity here."""
    l = np.asarray(logits, dtype=np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        top = l.max(1, keepdims=True)
        e = np.where(l == top, 1.0, np.exp(l - top)) * (l > -np.inf)
        total = e.sum(1, keepdims=True)
        return np.divide(e, total, out=np.zeros_like(e), where=total > 0)


def route_ref(logits, topk, bias=None, *, score="softmax", groups=1, topk_groups=1, group_top=1, renormalize=False,
              scale=1.0):
    """(weights float64 [M, topk], ids [M, topk]): one token at a time, by sorting."""
    l = np.asarray(logits, dtype=np.float64)
    M, E = l.shape
    s = scores_ref(l, score)
    group_top = group_top if groups > 1 else 1
    weights, ids = np.zeros((M, topk)), np.full((M, topk), -1, dtype=np.int32)
    per = E // groups
    for m in range(M):
        if bias is not None:
            key = s[m] + np.asarray(bias, dtype=np.float64)
        else:
            key = l[m].copy() if group_top == 1 else s[m].copy()
        key[~(l[m] > -np.inf) | ~(key > -np.inf)] = -np.inf
        if groups > 1:
            of = []
            for g in range(groups):
                best = sorted((k for k in key[g * per:(g + 1) * per] if k > -np.inf), reverse=True)[:group_top]
                of.append(sum(best) if best else -np.inf)
            order = sorted(range(groups), key=lambda g: (-of[g], g))[topk_groups:]
            for g in order:
                key[g * per:(g + 1) * per] = -np.inf
        left = [e for e in range(E) if key[e] > -np.inf]
        chosen = sorted(left, key=lambda e: (-key[e], e))[:topk]
        ids[m, :len(chosen)] = chosen
        w = s[m][chosen]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else 0.0 * w
        weights[m, :len(chosen)] = w * scale
        if np.isnan(l[m]).any():
            weights[m] = np.nan
    return weights, ids


def route_weights_ref(logits, ids, *, score, renormalize, scale):
    """The weights of a given choice: what route_backward_ref differentiates."""
    s = scores_ref(logits, score)
    E = s.shape[1]
    named = (ids >= 0) & (ids < E)
    p = np.take_along_axis(s, np.where(named, ids, 0), 1) * named
    if renormalize:
        total = p.sum(1, keepdims=True)
        p = np.divide(p, total, out=np.zeros_like(p), where=total > 0)
    return p * scale


def route_backward_ref(dweights, logits, ids, *, score, renormalize, scale):
    """(dlogits float64 [M, E], bound [M, E]): bound is the sum of the magnitudes that the
    formula adds, which rounding errors are relative to."""
    l, dw = np.asarray(logits, dtype=np.float64), np.asarray(dweights, dtype=np.float64) * scale
    M, E = l.shape
    s = scores_ref(l, score)
    rest = 1.0 / (1.0 + np.exp(np.where(np.isnan(l), 0, l)))
    out, bound = np.zeros((M, E)), np.zeros((M, E))
    for m in range(M):
        slots = [j for j in range(ids.shape[1]) if 0 <= ids[m, j] < E]
        p = s[m][ids[m, slots]]
        g, size = dw[m, slots], np.abs(dw[m, slots])
        if renormalize:
            total = p.sum()
            if total > 0:
                g, size = (g - (p * g).sum() / total) / total, (size + (p * size).sum() / total) / total
            else:
                g, size = 0 * g, 0 * size
        ds, dsize = np.zeros(E), np.zeros(E)
        np.add.at(ds, ids[m, slots], g)
        np.add.at(dsize, ids[m, slots], size)
        if score == "softmax":
            out[m] = s[m] * (ds - (s[m] * ds).sum())
            bound[m] = s[m] * (dsize + (s[m] * dsize).sum())
        else:
            out[m], bound[m] = ds * s[m] * rest[m], dsize * s[m] * rest[m]
        if np.isnan(l[m]).any():
            out[m] = np.nan
    return out, bound


# --------------------------------------------------------------- e4m3 ---

def e4m3_values() -> np.ndarray:
    """The 256 codes' values in float64 (0x7F and 0xFF: NaN)."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8.0 + f) * 2.0 ** (e - 10.0), f * 2.0 ** -9.0)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


def to_e4m3(v) -> np.ndarray:
    """Codes of float64 values of magnitude at most 448, to nearest-even; others and NaN become NaN codes."""
    v = np.asarray(v, dtype=np.float64)
    table = e4m3_values()[:127]
    mag = np.abs(v)
    with np.errstate(invalid="ignore"):
        fine = mag <= 448
    at = np.searchsorted(table, np.where(fine, mag, 0), side="right") - 1
    up = np.minimum(at + 1, 126)
    low, high, x = table[at], table[up], np.where(fine, mag, 0)
    middle = (low + high) / 2
    code = np.where((x > middle) | ((x == middle) & (up % 2 == 0) & (up > at)), up, at)
    code = np.where(fine, code, 127)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def fp8_quantize_ref(x):
    """(codes uint8 [M, K'], scales uint8 [M, B]) of float64 x [M, K]."""
    x = np.asarray(x, dtype=np.float64)
    M, K = x.shape
    blocks, B = (K + 127) // 128, (K + 511) // 512 * 4
    codes, scales = np.zeros((M, blocks * 128), dtype=np.uint8), np.full((M, B), 127, dtype=np.uint8)
    for b in range(blocks):
        part = x[:, 128 * b:128 * (b + 1)]
        top = np.abs(np.where(np.isfinite(part), part, 0)).max(1)
        e = np.zeros(M, dtype=np.int64)
        for m in np.nonzero(top)[0]:
            while 448.0 * 2.0 ** e[m] < top[m]:
                e[m] += 1
            while e[m] > -126 and 448.0 * 2.0 ** (e[m] - 1.0) >= top[m]:
                e[m] -= 1
        codes[:, 128 * b:128 * b + part.shape[1]] = to_e4m3(part / 2.0 ** e[:, None])
        scales[:, b] = e + 127
    return codes, scales


def spread(scales, rows, cols):
    """Block scales [ceil(rows / 128), ceil(cols / 128)] for every element."""
    return np.repeat(np.repeat(np.asarray(scales, dtype=np.float64), 128, 0)[:rows], 128, 1)[:, :cols]


def fp8_linear_ref(codes, scales, w, ws, K: int, transpose: bool):
    """(y [M, N] float64, slack [M, N]) of codes [M, K'] with e8m0 scales [M, B] and weight codes
    w (uint8; [N, K], or [K, N] transposed) with float64 block scales ws.

    slack: how far the matrix unit's sums may lie off.  It drops, of each product among eight
    neighbouring k, what lies more than 13 bits below the largest exponent among them (exponents
    of the codes' fields added; one bit more where a product of mantissas reaches 2), and adds in
    fp32: 2^-24 of the magnitudes for each of the K / 8 sums and the additions behind them."""
    table = e4m3_values()
    wt = w if transpose else w.T                      # [K, N]
    W = table[wt] * (spread(ws, *w.shape) if transpose else spread(ws, *w.shape).T)
    xv = table[codes[:, :K]]
    xs = np.repeat(2.0 ** (scales.astype(np.float64) - 127), 128, 1)[:, :K]
    y = (xv * xs) @ W
    M, N = y.shape
    field = lambda c: np.maximum((c.astype(np.int64) >> 3) & 15, 1) - 7  # noqa: E731
    pad = -K % 8
    ex = np.pad(field(codes[:, :K]), ((0, 0), (0, pad)), constant_values=-6)
    ew = np.pad(field(wt), ((0, pad), (0, 0)), constant_values=-6)
    drop = np.zeros((M, N))
    wabs, sabs = np.abs(table[wt]), np.abs(spread(ws, *w.shape) if transpose else spread(ws, *w.shape).T)
    for o in range(0, K, 8):
        hi = min(o + 8, K)
        top = (ex[:, o:o + 8, None] + ew[None, o:o + 8, :]).max(1)
        p = np.abs(xv[:, o:hi, None]) * wabs[None, o:hi, :]
        unit = 2.0 ** (top - 12.0)
        lost = np.where(p % (unit[:, None, :] / 2) == 0, 0.0, np.minimum(p, unit[:, None, :])).sum(1)
        drop += lost * xs[:, o, None] * sabs[None, o, :]
    total = (np.abs(xv) * xs) @ (wabs * sabs)
    return y, drop + 2.0 ** -24 * (K / 8 + 16) * total
