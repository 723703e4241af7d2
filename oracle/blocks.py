"""fp64 definitions of the RMS norm, the e4m3 block quantizer and grouped products.

Block quantizer: a = max(max|x|, 2^-100) over a block (1 x 128 of a row, 128 x 128 of a
weight, short at the edges), scale = fp32(a / 448), code value = e4m3 nearest-even of the
real quotient 448 x / a. A block with a NaN or an infinity has NaN codes.
"""
from __future__ import annotations

import numpy as np

FLOOR = 2.0 ** -100
E4M3_MAX = 448.0


def e4m3_round(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value (ties to even) of |v| <= 448, from the format: quantum 2^(e-3), at least 2^-9."""
    v = np.asarray(v, np.float64)
    _, e = np.frexp(v)
    q = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.rint(v / q) * q


def _exact_quotient_round(x: np.ndarray, a: np.ndarray) -> np.ndarray:
    """e4m3_round of the real 448 x / a. The fp64 quotient of an fp32 x and a decides right: it is
    exact wherever the real quotient is a midpoint (few bits), and a quotient that is no
    midpoint differs from one by more than an fp64 ulp."""
    return e4m3_round(448.0 * x / a)


def quantize_rows(x: np.ndarray):
    """(code values fp64 [M, in], scales fp32 [M, nb]) of rows x."""
    x = np.asarray(x, np.float64)
    M, n = x.shape
    nb = -(-n // 128)
    q = np.empty_like(x)
    s = np.empty((M, nb), np.float32)
    for b in range(nb):
        blk = x[:, b * 128:(b + 1) * 128]
        bad = ~np.isfinite(blk).all(1)
        with np.errstate(invalid="ignore"):
            a = np.maximum(np.abs(blk).max(1), FLOOR)
            q[:, b * 128:(b + 1) * 128] = _exact_quotient_round(blk, a[:, None])
        q[bad, b * 128:(b + 1) * 128] = np.nan
        s[:, b] = (a.astype(np.float32) / np.float32(448))
    return q, s


def quantize_weight(W: np.ndarray):
    """(code values fp64, scales fp32) of one weight [out, in]."""
    W = np.asarray(W, np.float64)
    o, i = W.shape
    q = np.empty_like(W)
    s = np.empty((-(-o // 128), -(-i // 128)), np.float32)
    for r in range(s.shape[0]):
        for c in range(s.shape[1]):
            blk = W[r * 128:(r + 1) * 128, c * 128:(c + 1) * 128]
            if not np.isfinite(blk).all():
                q[r * 128:(r + 1) * 128, c * 128:(c + 1) * 128] = np.nan
                s[r, c] = np.nan if np.isnan(blk).any() else np.inf
                continue
            a = max(np.abs(blk).max(), FLOOR)
            q[r * 128:(r + 1) * 128, c * 128:(c + 1) * 128] = _exact_quotient_round(blk, a)
            s[r, c] = np.float32(a) / np.float32(448)
    return q, s


def row_values(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    return q * np.repeat(s.astype(np.float64), 128, 1)[:, : q.shape[1]]


def weight_values(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    up = np.repeat(np.repeat(s.astype(np.float64), 128, 0), 128, 1)
    return q * up[: q.shape[0], : q.shape[1]]


def rms_norm(h: np.ndarray, w: np.ndarray, eps: float):
    """(y, rstd) of rows h in fp64."""
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * w, rstd


def rms_norm_backward(dy: np.ndarray, h: np.ndarray, w: np.ndarray, eps: float, dh=None):
    """(dx, dw): gradients of sum(y dy) + sum(h dh)."""
    _, rstd = rms_norm(h, w, eps)
    n = h * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - n * (g * n).mean(1, keepdims=True))
    return dx if dh is None else dx + dh, (dy * n).sum(0)


def spans(offsets) -> list:
    return list(zip(offsets[:-1], offsets[1:]))


def grouped_forward(X, Ws, offsets):
    """Y [M, out], NaN outside every group."""
    Y = np.full((X.shape[0], Ws[0].shape[0]), np.nan)
    for e, (a, b) in enumerate(spans(offsets)):
        Y[a:b] = X[a:b] @ Ws[e].T
    return Y


def grouped_backward(X, dY, Ws, offsets):
    """(dX with NaN outside every group, dW [E, out, in])."""
    dX = np.full((dY.shape[0], Ws[0].shape[1]), np.nan)
    dW = np.zeros((len(Ws),) + Ws[0].shape)
    for e, (a, b) in enumerate(spans(offsets)):
        dX[a:b] = dY[a:b] @ Ws[e]
        if X is not None:
            dW[e] = dY[a:b].T @ X[a:b]
    return dX, dW
