"""Pins of the fp64 definitions of the RMS norm, the e4m3 block quantizer and grouped products."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import blocks, nf4


def test_e4m3_round_is_the_nearest_of_all_codes():
    table = nf4.e4m3_decode(np.arange(256, dtype=np.uint8)).astype(np.float64)
    pos = np.sort(table[:127])
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-448, 448, 4000), rng.uniform(-2.0 ** -5, 2.0 ** -5, 4000), pos, -pos,
                        (pos[1:] + pos[:-1]) / 2])
    got = blocks.e4m3_round(v)
    for x, g in zip(v, got):
        d = np.abs(pos - abs(x))
        near = np.flatnonzero(d == d.min())
        assert abs(g) == pos[near[0]] if len(near) == 1 else abs(g) == pos[near[near % 2 == 0][0]]
    assert np.array_equal(got, torch.tensor(v, dtype=torch.float32).to(torch.float8_e4m3fn).double().numpy())


def test_quantizer_decides_by_the_real_quotient():
    """Against exact rationals, for every pair of significands that makes a tie and some that do not."""
    rng = np.random.default_rng(1)
    pos = np.sort(nf4.e4m3_decode(np.arange(127, dtype=np.uint8)).astype(np.float64))
    mids = [(Fraction(float(pos[k])) + Fraction(float(pos[k + 1]))) / 2 for k in range(126)]
    for _ in range(300):
        a = int(rng.integers(128, 256))
        x = int(rng.integers(1, a + 1))
        row = np.zeros((1, 128))
        row[0, 0], row[0, 1] = a, x
        q, s = blocks.quantize_rows(row)
        t = Fraction(448 * x, a)
        above = sum(1 for m in mids if t > m)
        tie = t in mids
        k = above + (1 if tie and above % 2 == 1 else 0)
        assert q[0, 1] == pos[k] and q[0, 0] == 448 and s[0, 0] == np.float32(a) / np.float32(448)


def test_planted_mistakes_in_the_quantizer_are_seen():
    """A quotient formed as x * fp32(448 / a) rounds some ties the wrong way."""
    x = np.arange(1, 256, dtype=np.float64)
    wrong = 0
    for a in range(128, 256):
        v = x[x <= a]
        inv = np.float32(448) / np.float32(a)
        wrong += int((blocks.e4m3_round((v.astype(np.float32) * inv).astype(np.float64)) !=
                      blocks.e4m3_round(448 * v / a)).sum())
    assert wrong > 0


def test_zero_and_short_blocks():
    q, s = blocks.quantize_rows(np.zeros((2, 130)))
    assert not q.any() and s.shape == (2, 2) and (s == np.float32(2.0 ** -100) / np.float32(448)).all()
    q, s = blocks.quantize_weight(np.ones((130, 129)))
    assert s.shape == (2, 2) and (q == 448).all()
    assert np.allclose(blocks.weight_values(q, s), 1, rtol=2.0 ** -23)


@pytest.mark.parametrize("with_dh", [True, False])
def test_norm_backward_against_differences(with_dh):
    rng = np.random.default_rng(2)
    h, w, dy = rng.normal(size=(3, 11)), rng.normal(size=11), rng.normal(size=(3, 11))
    dh = rng.normal(size=(3, 11)) if with_dh else None

    def f(h, w):
        return (blocks.rms_norm(h, w, 1e-3)[0] * dy).sum() + (0 if dh is None else (h * dh).sum())

    dx, dw = blocks.rms_norm_backward(dy, h, w, 1e-3, dh)
    eps = 1e-6
    for idx in np.ndindex(h.shape):
        d = np.zeros_like(h)
        d[idx] = eps
        assert abs((f(h + d, w) - f(h - d, w)) / (2 * eps) - dx[idx]) < 1e-8 * max(1, abs(dx[idx]))
    for j in range(11):
        d = np.zeros_like(w)
        d[j] = eps
        assert abs((f(h, w + d) - f(h, w - d)) / (2 * eps) - dw[j]) < 1e-8 * max(1, abs(dw[j]))


def test_grouped_backward_against_differences():
    rng = np.random.default_rng(3)
    off = [1, 3, 3, 6]
    X, G = rng.normal(size=(7, 4)), rng.normal(size=(7, 5))
    Ws = [rng.normal(size=(5, 4)) for _ in range(3)]

    def f(X, Ws):
        return np.nansum(blocks.grouped_forward(X, Ws, off) * G)

    dX, dW = blocks.grouped_backward(X, G, Ws, off)
    eps = 1e-6
    for idx in np.ndindex(X.shape):
        d = np.zeros_like(X)
        d[idx] = eps
        g = (f(X + d, Ws) - f(X - d, Ws)) / (2 * eps)
        assert abs(g - (0 if np.isnan(dX[idx]) else dX[idx])) < 1e-7
    for e in range(3):
        for idx in np.ndindex(5, 4):
            up = [w.copy() for w in Ws]
            dn = [w.copy() for w in Ws]
            up[e][idx] += eps
            dn[e][idx] -= eps
            assert abs((f(X, up) - f(X, dn)) / (2 * eps) - dW[e][idx]) < 1e-7
