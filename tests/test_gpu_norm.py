"""GPU parity: RMS norm with residual, bf16 and e4m3 output, and its backward against fp64."""
import numpy as np
import pytest
import torch

from oracle import blocks
from quantized_lora_fine_b200 import api
from tests.block_helpers import U_BF16, U_F32, bf16_round, f64, normal, outliers

pytestmark = pytest.mark.gpu

EPS = 1e-6
SHAPES = [(1, 8), (1, 4096), (3, 16), (5, 136), (33, 256), (129, 520), (17, 1024), (64, 5120), (9, 8192), (3, 11008),
          (2, 16384), (2, 32768), (700, 264)]


def rel_fwd(H):
    """Relative error of rstd and, with two more products, of the fp32 y: a sum of H squares (each rounded,
    all of one sign) is off by H + 1 half-steps at most and the root halves that; division, + eps, root,
    division, and the two products: 8 more are plenty."""
    return ((H + 1) / 2 + 8) * U_F32


def _case(M, H, residual, wdtype, seed):
    x = outliers((M, H), seed)
    r = outliers((M, H), seed + 1) if residual else None
    w = (1 + 0.2 * normal((H,), seed + 2).float()).to(wdtype)
    h = f64(x) if r is None else bf16_round(f64(x) + f64(r))
    return x, r, w, h


@pytest.mark.parametrize("M,H", SHAPES)
@pytest.mark.parametrize("residual,wdtype", [(True, torch.bfloat16), (False, torch.float32)])
def test_forward_bf16(cuda_device, M, H, residual, wdtype):
    x, r, w, h = _case(M, H, residual, wdtype, M + H)
    dx, dr, dw = (None if t is None else t.to(cuda_device) for t in (x, r, w))
    y, hh, rstd = api.rms_norm_fwd(dx, dw, EPS, residual=dr)
    yr, rr = blocks.rms_norm(h, f64(w), EPS)
    assert np.array_equal(f64(hh), h)
    assert (hh.data_ptr() == dx.data_ptr()) == (not residual)
    assert np.all(np.abs(f64(rstd) - rr) <= rel_fwd(H) * rr)
    d = rel_fwd(H)
    assert np.all(np.abs(f64(y) - yr) <= (U_BF16 * (1 + d) + d) * np.abs(yr) + 2.0 ** -134)


@pytest.mark.parametrize("M,H", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_forward_fp8(cuda_device, M, H, residual):
    x, r, w, h = _case(M, H, residual, torch.bfloat16, M + H + 5)
    q, hh, rstd = api.rms_norm_fwd(x.to(cuda_device), w.to(cuda_device), EPS,
                                   residual=None if r is None else r.to(cuda_device), fp8=True)
    y, _ = blocks.rms_norm(h, f64(w), EPS)
    assert np.array_equal(f64(hh), h)
    _, s = blocks.quantize_rows(y)
    d = rel_fwd(H)
    assert np.all(np.abs(f64(q.scale) - s) <= (d + 2 * U_F32) * s)
    # the real quotient, and how far the fp32 one (two values of relative error d, the quotient's own) may be
    nb = s.shape[1]
    pad = np.pad(np.abs(y), ((0, 0), (0, nb * 128 - H))).reshape(M, nb, 128).max(2)
    t = 448 * y / np.repeat(np.maximum(pad, blocks.FLOOR), 128, 1)[:, :H]
    half = np.exp2(np.floor(np.log2(np.maximum(np.abs(t), 2.0 ** -6))) - 4)
    assert np.all(np.abs(f64(q.codes) - t) <= half * (1 + 2.0 ** -20) + (2 * d + 4 * U_F32) * np.abs(t))


@pytest.mark.parametrize("M,H", SHAPES + [(1500, 256)])
@pytest.mark.parametrize("dh,wdtype", [(True, torch.bfloat16), (False, torch.float32)])
def test_backward(cuda_device, M, H, dh, wdtype):
    x, _, w, h = _case(M, H, False, wdtype, M + H + 9)
    dy = normal((M, H), M + 3)
    g = normal((M, H), M + 4) if dh else None
    _, hh, rstd = api.rms_norm_fwd(x.to(cuda_device), w.to(cuda_device), EPS)
    args = (dy.to(cuda_device), hh, rstd, w.to(cuda_device))
    dx, dw = api.rms_norm_bwd(*args, dh=None if g is None else g.to(cuda_device))
    W = f64(w)
    dxr, dwr = blocks.rms_norm_backward(f64(dy), h, W, EPS, None if g is None else f64(g))
    _, rr = blocks.rms_norm(h, W, EPS)
    n = np.abs(h) * rr[:, None]
    gg = np.abs(f64(dy) * W)
    # every term in fp32 from an rstd of relative error d (at most cubed); a mean of H terms
    d = 4 * rel_fwd(H) + (H + 8) * U_F32
    terms = rr[:, None] * (gg + n * (gg * n).mean(1, keepdims=True)) + (0 if g is None else np.abs(f64(g)))
    assert np.all(np.abs(f64(dx) - dxr) <= U_BF16 * np.abs(dxr) + (1 + U_BF16) * d * terms + 2.0 ** -134)
    assert np.all(np.abs(f64(dw) - dwr) <= (rel_fwd(H) + (M + 4) * U_F32) * (np.abs(f64(dy)) * n).sum(0) + 2.0 ** -149)
    dx2, none = api.rms_norm_bwd(*args, dh=None if g is None else g.to(cuda_device), need_dw=False)
    assert none is None and torch.equal(dx2, dx)
    _, dw2 = api.rms_norm_bwd(*args)
    assert torch.equal(dw2, dw)       # the same bits from run to run


def test_zero_rows(cuda_device):
    """A row of zeros gives zeros (eps keeps rstd finite), in 8 bit too."""
    x = normal((4, 256), 1)
    x[2] = 0
    w = torch.ones(256, dtype=torch.bfloat16, device=cuda_device)
    y, _, rstd = api.rms_norm_fwd(x.to(cuda_device), w, EPS)
    q, _, _ = api.rms_norm_fwd(x.to(cuda_device), w, EPS, fp8=True)
    assert not y[2].any() and not q.codes[2].float().any() and torch.isfinite(q.scale).all()
    assert abs(float(rstd[2]) - 1000) < 1e-3


def test_nan_rows_stay_in_their_rows(cuda_device):
    x = normal((5, 512), 2)
    clean = api.rms_norm_fwd(x.to(cuda_device), torch.ones(512, dtype=torch.bfloat16, device=cuda_device), EPS)[0]
    x[1, 7] = float("nan")
    x[3, 500] = float("inf")
    y = api.rms_norm_fwd(x.to(cuda_device), torch.ones(512, dtype=torch.bfloat16, device=cuda_device), EPS)[0]
    assert torch.isnan(y[1]).all()
    assert torch.equal(y[[0, 2, 4]], clean[[0, 2, 4]])
