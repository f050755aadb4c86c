"""The MX-matrix and router-training operators in plain float64 (oracle; test
infrastructure only, no code shared with the library).

Formats, block scales and layouts are the MX mode's (oracle/mx.py); here also
the E2M1 encoder, non-finite blocks, the product of quantised rows with MXFP4
matrices, the router's load and losses, and their gradients.
"""
from __future__ import annotations

import numpy as np

from . import mx

FP4, FP8 = 0, 1


def e2m1_encode(v: np.ndarray) -> np.ndarray:
    """float64 values -> E2M1 codes: nearest magnitude of 0, 0.5, 1, 1.5, 2, 3, 4,
    6, ties to the even code, past 6 saturated; the sign bit is v's."""
    a = np.abs(np.asarray(v, dtype=np.float64))
    grid = mx.e2m1_to_f64(np.arange(8))
    mids = (grid[1:] + grid[:-1]) / 2
    low = np.searchsorted(mids, a, side="left")        # at a midpoint: the lower code
    up = low + ((low % 2 == 1) & (a == mids[np.minimum(low, 6)]))
    return (up | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def quantize(v: np.ndarray, fmt: int):
    """Rows [..., K] -> (codes [..., K] one per element, E8M0 bytes [..., K/32])."""
    v = np.asarray(v, dtype=np.float64)
    b = v.reshape(v.shape[:-1] + (v.shape[-1] // 32, 32))
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    e = np.frexp(amax)[1] - 1                            # floor(log2), exact
    x = np.where(amax > 0, np.clip(e - (2 if fmt == FP4 else 8) + 127, 0, 254), 0)
    a = b / np.exp2(x - 127.0)[..., None]
    codes = e2m1_encode(a) if fmt == FP4 else mx.e4m3_encode(a)
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8)
    return codes.reshape(v.shape), np.where(bad, 255, x).astype(np.uint8)


def values(codes: np.ndarray, x: np.ndarray, fmt: int) -> np.ndarray:
    """The values of codes [..., K] with E8M0 bytes [..., K/32]."""
    c = mx.e2m1_to_f64(codes) if fmt == FP4 else mx.e4m3_to_f64(codes)
    return c * np.repeat(mx.e8m0_to_f64(x), 32, axis=-1)


def rounded(v: np.ndarray, fmt: int) -> np.ndarray:
    """The values v's rows take in the format."""
    return values(*quantize(v, fmt), fmt)


def pack(codes: np.ndarray, fmt: int) -> np.ndarray:
    """Stored bytes of codes [..., K]: E2M1 two a byte, element 2i in the low nibble."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4) if fmt == FP4 else codes


def by_step(x: np.ndarray) -> np.ndarray:
    """E8M0 bytes [M, N, K/32] -> the stored [M, K/128, N, 4]."""
    M, N, nb = x.shape
    return np.ascontiguousarray(x.reshape(M, N, nb // 4, 4).transpose(0, 2, 1, 3))


def product(x: np.ndarray, fmt: int, W: np.ndarray, offsets=None, row_src=None, R=None):
    """Rows of x [T][K] rounded to fmt, times the matrices W [M][N][K] (float64
    values).  Returns (y [R][N], the magnitude sums of its products [R][N]);
    rows of no matrix are NaN."""
    q = rounded(x, fmt)
    R = (len(x) if row_src is None else len(row_src)) if R is None else R
    src = np.arange(R) if row_src is None else np.asarray(row_src)
    rows = np.where(((src >= 0) & (src < len(x)))[:, None], q[np.clip(src, 0, len(x) - 1)], 0.0)
    off = np.array([0, R]) if offsets is None else np.asarray(offsets)
    y = np.full((R, W.shape[1]), np.nan)
    mag = np.full((R, W.shape[1]), np.nan)
    for m in range(len(off) - 1):
        s = slice(off[m], off[m + 1])
        if off[m + 1] > off[m]:
            y[s] = rows[s] @ W[m].T
            mag[s] = np.abs(rows[s]) @ np.abs(W[m]).T
    return y, mag


# ------------------------------------------------------------------ the router ----

def _softmax(z):
    """Rows of logits -> (probabilities, log sum exp); a row of -inf alone: zeros."""
    m = z.max(1, keepdims=True)
    b = np.where(np.isneginf(m), 0.0, m)
    e = np.exp(z - b)
    n = e.sum(1, keepdims=True)
    none = n == 0
    return np.where(none, 0.0, e / np.where(none, 1, n)), np.where(none, 0.0, b + np.log(np.where(none, 1, n)))[:, 0]


def _seqs(T, offsets):
    off = [0, T] if offsets is None else [int(v) for v in offsets]
    return list(zip(off[:-1], off[1:]))


def balance(logits, topk_idx, offsets=None):
    """(counts [S][E], mean probabilities [S][E], [balance loss, z loss])."""
    z = np.asarray(logits, dtype=np.float64)
    (T, E), k = z.shape, topk_idx.shape[1]
    p, lse = _softmax(z)
    seqs = _seqs(T, offsets)
    counts = np.zeros((len(seqs), E), dtype=np.int64)
    probs = np.zeros((len(seqs), E))
    per_seq, z2 = [], []
    for s, (lo, hi) in enumerate(seqs):
        if hi <= lo:
            continue
        ids = topk_idx[lo:hi].reshape(-1)
        counts[s] = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
        probs[s] = p[lo:hi].mean(0)
        per_seq.append(float(E / (k * (hi - lo)) * counts[s] @ probs[s]))
        z2.extend(lse[lo:hi] ** 2)
    return counts, probs, np.array([np.mean(per_seq) if per_seq else 0.0, np.mean(z2) if z2 else 0.0])


def route_backward(logits, topk_idx, topk_w=None, d_topk_w=None, d_loss=None, counts=None, offsets=None):
    """(dz [T][E], the magnitudes of the terms it is summed from [T][E])."""
    z = np.asarray(logits, dtype=np.float64)
    T, E = z.shape
    k = topk_idx.shape[1]
    dz, mag = np.zeros((T, E)), np.zeros((T, E))
    if d_topk_w is not None:
        w, dw = np.asarray(topk_w, np.float64), np.asarray(d_topk_w, np.float64)
        v = w * (dw - (w * dw).sum(1, keepdims=True))
        a = np.abs(w) * (np.abs(dw) + np.abs(w * dw).sum(1, keepdims=True))
        for j in range(k):
            t = np.nonzero((topk_idx[:, j] >= 0) & (topk_idx[:, j] < E))[0]
            np.add.at(dz, (t, topk_idx[t, j]), v[t, j])
            np.add.at(mag, (t, topk_idx[t, j]), a[t, j])
    if d_loss is not None:
        p, lse = _softmax(z)
        seqs = _seqs(T, offsets)
        live = sum(hi > lo for lo, hi in seqs)
        n = sum(max(hi - lo, 0) for lo, hi in seqs)
        gb, gz = (float(v) for v in d_loss)
        for s, (lo, hi) in enumerate(seqs):
            if hi <= lo:
                continue
            f = np.asarray(counts[s], np.float64) * E / (k * (hi - lo))
            q = p[lo:hi]
            mean = (q @ f)[:, None]
            dz[lo:hi] += gb / live / (hi - lo) * q * (f - mean) + 2 * gz / n * lse[lo:hi, None] * q
            mag[lo:hi] += abs(gb) / live / (hi - lo) * q * (f + mean) + 2 * abs(gz) / n * np.abs(lse[lo:hi, None]) * q
    return dz, mag
