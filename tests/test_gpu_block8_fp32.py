"""e4m3 codes of fp32 values. Weights: of the real quotient 448 x / a, bit for bit, also where it lies within an fp32
rounding of the midpoint of two codes. The norm's y: of the quotient rounded to fp32."""
import bisect
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import blocks, nf4
from quantized_lora_fine_b200 import api
from tests.block_helpers import f64, normal, outliers

CODES = np.sort(nf4.e4m3_decode(np.arange(127, dtype=np.uint8)).astype(np.float64))
MIDS = (CODES[1:] + CODES[:-1]) / 2


def near_midpoints(n: int, seed: int) -> np.ndarray:
    """fp32 [n, 128]: each row a block with its maximum first, a random fp32, and for every midpoint m of two codes
    one of the fp32 values around m a / 448."""
    rng = np.random.default_rng(seed)
    a = np.ldexp(rng.integers(1 << 23, 1 << 24, n).astype(np.float64), rng.integers(-60, 20, n))
    x = (MIDS[None, :] * a[:, None] / 448).astype(np.float32)
    x = (x.view(np.int32) + rng.integers(-2, 3, x.shape, dtype=np.int32)).view(np.float32)
    x *= rng.choice(np.array([-1, 1], np.float32), x.shape)
    x = np.minimum(np.abs(x), a[:, None].astype(np.float32)) * np.sign(x)
    return np.concatenate([a[:, None].astype(np.float32), x, np.zeros((n, 1), np.float32)], 1)


def test_the_oracle_decides_fp32_values_by_the_real_quotient():
    x = near_midpoints(40, 0)
    q, _ = blocks.quantize_rows(x.astype(np.float64))
    mids = [Fraction(float(m)) for m in MIDS]
    for row, got in zip(x, q):
        a = Fraction(float(row[0]))
        for v, g in zip(row, got):
            t = abs(448 * Fraction(float(v)) / a)
            k = bisect.bisect_left(mids, t)                   # midpoints below t
            if k < len(mids) and mids[k] == t and k % 2 == 1:
                k += 1                                        # (a tie: to the even code)
            assert abs(g) == CODES[k], (float(v), float(row[0]))


def _same(got: torch.Tensor, want: np.ndarray, name):
    g = f64(got)
    bad = g != want
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size} differ, first {g[bad][0]} for {want[bad][0]}"


def _weight_of(rows: np.ndarray) -> np.ndarray:
    """[n, 128] blocks' values as a weight whose 128 x 128 blocks hold one block's values each, shuffled."""
    rng = np.random.default_rng(5)
    n = rows.shape[0]
    w = np.zeros((128 * n, 128), np.float32)
    for b in range(n):
        at = rng.permutation(128 * 128)[:128]
        w[128 * b:128 * (b + 1)].reshape(-1)[at] = rows[b]
    return w


@pytest.mark.gpu
def test_one_weight_just_off_a_midpoint(cuda_device):
    W = np.zeros((128, 128), np.float32)
    W[0, 0], W[77, 5] = float.fromhex("0x1.ff2344p+1"), float.fromhex("0x1.a3dcf6p-2")
    w = api.fp8_quantize_weight(torch.from_numpy(W).to(cuda_device))
    assert float(w.codes[77, 5].float()) == 44 and float(w.codes[0, 0].float()) == 448


@pytest.mark.gpu
def test_weights_near_midpoints(cuda_device):
    W = _weight_of(near_midpoints(300, 1))
    w = api.fp8_quantize_weight(torch.from_numpy(W).to(cuda_device))
    codes, scale = blocks.quantize_weight(W.astype(np.float64))
    _same(w.codes, codes, "codes")
    _same(w.scale, scale, "scale")
    assert api.status() == 0


@pytest.mark.gpu
def test_weights_of_extreme_size(cuda_device):
    """Blocks at both ends of fp32, subnormals, zeros, blocks below the floor, a single NaN and infinity."""
    rng = np.random.default_rng(2)
    W = rng.normal(size=(8, 128, 128)).astype(np.float32)
    W[0] *= np.float32(1e37)
    W[1] = np.ldexp(rng.integers(-(1 << 23), 1 << 23, (128, 128)), -149).astype(np.float32)
    W[2] = 0
    W[3] = np.float32(3.4028235e38)
    W[4] *= np.float32(2.0 ** -101)
    W[5, 3, 4] = np.nan
    W[6, 100, 1] = np.inf
    W = W.reshape(-1, 128)
    w = api.fp8_quantize_weight(torch.from_numpy(W).to(cuda_device))
    codes, scale = blocks.quantize_weight(W.astype(np.float64))
    assert np.array_equal(f64(w.codes), codes, equal_nan=True)
    assert np.array_equal(f64(w.scale), scale.astype(np.float64), equal_nan=True)
    assert api.status() == 8          # QLORA_ERR_NONFINITE
    api.reset_status(api.Workspace.status_word(0))


@pytest.mark.gpu
@pytest.mark.parametrize("M,H,wdtype", [(400, 4096, torch.bfloat16), (400, 5120, torch.float32), (7, 264, torch.bfloat16)])
def test_norm_output_is_quantized_from_its_fp32_value(cuda_device, M, H, wdtype):
    """y = (h rstd) w, each product rounded to fp32, from the rstd that the call returns; the quotient rounded to
    fp32 decides: 448 y / a is off by two half places of u = 448 p y and one of t, 2^-22 in all, and within that
    of a midpoint either neighbour may come out, elsewhere the real quotient's code."""
    x = outliers((M, H), M)
    w = (1 + 0.2 * normal((H,), 3).float()).to(wdtype)
    q, h, rstd = api.rms_norm_fwd(x.to(cuda_device), w.to(cuda_device), 1e-6, fp8=True)
    y = f64(h).astype(np.float32) * f64(rstd).astype(np.float32)[:, None] * f64(w).astype(np.float32)
    y = y.astype(np.float64)
    codes, scale = blocks.quantize_rows(y)
    _same(q.scale, scale, "scale")
    got = f64(q.codes)
    a = np.repeat(np.maximum(blocks_max(y), blocks.FLOOR), 128, 1)[:, :H]
    t = 448 * np.abs(y) / a
    lo, hi = blocks.e4m3_round(t * (1 - 2.0 ** -22)), blocks.e4m3_round(np.minimum(t * (1 + 2.0 ** -22), 448))
    assert ((lo <= np.abs(got)) & (np.abs(got) <= hi) & (np.sign(got) * np.sign(y) >= 0)).all()
    assert (got == codes)[lo == hi].all()


def blocks_max(y: np.ndarray) -> np.ndarray:
    M, H = y.shape
    nb = -(-H // 128)
    return np.pad(np.abs(y), ((0, 0), (0, nb * 128 - H))).reshape(M, nb, 128).max(2)
