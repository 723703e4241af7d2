"""GPU parity: e4m3 block quantizers (bit for bit) and the 8-bit linear against fp64."""
import numpy as np
import pytest
import torch

from oracle import blocks
from quantized_lora_fine_b200 import api
from tests.block_helpers import assert_product, f64, normal, outliers

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status(cuda_device):
    yield
    torch.cuda.synchronize()
    assert api.status() == 0


def _same(got: torch.Tensor, want: np.ndarray, name):
    g = f64(got)
    assert np.array_equal(np.isnan(g), np.isnan(want)), name
    ok = (g == want) | np.isnan(want)
    assert ok.all(), f"{name}: {int((~ok).sum())} differ, first at {np.argwhere(~ok)[0].tolist()}"


@pytest.mark.parametrize("M,n", [(1, 16), (3, 128), (5, 144), (64, 256), (129, 4096), (2, 11008), (333, 272), (7, 2032)])
def test_quantize_rows(cuda_device, M, n):
    x = outliers((M, n), seed=M + n)
    q = api.fp8_quantize_rows(x.to(cuda_device))
    codes, scale = blocks.quantize_rows(f64(x))
    _same(q.codes, codes, "codes")
    _same(q.scale, scale, "scale")


def test_quantize_rows_ties_and_extremes(cuda_device):
    """Every bf16 magnitude ratio of two significands against a block's maximum (ties among them),
    zero rows, subnormals, the largest and smallest values."""
    sig = torch.arange(128, 256, dtype=torch.float32)
    rows = []
    for a in range(128, 256):
        for e in (0, -3, -9, -14):
            r = sig * 2.0 ** e
            r = torch.where(r > a, r / 2, r)
            r[0] = a
            rows.append(r)
    x = torch.stack(rows)
    x = torch.cat([x, x * 2.0 ** -130, x * 2.0 ** 119, torch.zeros(3, 128), torch.full((1, 128), 2.0 ** -133),
                   torch.full((1, 128), 2.0 ** -100), torch.full((1, 128), 3.3e38)]).to(torch.bfloat16)
    q = api.fp8_quantize_rows(x.to(cuda_device))
    codes, scale = blocks.quantize_rows(f64(x))
    _same(q.codes, codes, "codes")
    _same(q.scale, scale, "scale")


def test_quantize_rows_nonfinite_blocks(cuda_device):
    x = normal((6, 400), 3)
    x[1, 5] = float("nan")
    x[2, 130] = float("inf")
    x[4, 399] = float("-inf")
    q = api.fp8_quantize_rows(x.to(cuda_device))
    codes, _ = blocks.quantize_rows(f64(x))
    _same(q.codes, codes, "codes")
    assert np.isnan(f64(q.scale)[1, 0]) and np.isinf(f64(q.scale)[2, 1]) and np.isinf(f64(q.scale)[4, 3])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(16, 16), (128, 128), (272, 400), (3, 144, 272), (2, 1024, 512)])
def test_quantize_weight(cuda_device, dtype, shape):
    W = torch.randn(shape, generator=torch.Generator().manual_seed(7)).mul_(0.02).to(dtype)
    w = api.fp8_quantize_weight(W.to(cuda_device))
    Ws, cs, ss = W.reshape(-1, *shape[-2:]), w.codes.reshape(-1, *shape[-2:]), w.scale.reshape(-1, *w.scale.shape[-2:])
    for e in range(Ws.shape[0]):
        codes, scale = blocks.quantize_weight(f64(Ws[e]))
        _same(cs[e], codes, "codes")
        _same(ss[e], scale, "scale")


def test_quantize_weight_reports_nonfinite(cuda_device):
    W = normal((256, 256), 1)
    W[200, 3] = float("inf")
    w = api.fp8_quantize_weight(W.to(cuda_device))
    torch.cuda.synchronize()
    assert api.status() == 8          # QLORA_ERR_NONFINITE
    api.reset_status(api.Workspace.status_word(0))
    assert torch.isnan(w.codes[128:, :128].float()).all() and not torch.isnan(w.codes[:128].float()).any()


def _weight(o, i, seed, dev):
    w = api.fp8_quantize_weight(normal((o, i), seed, 0.02, index=9).to(dev))
    return w, blocks.weight_values(f64(w.codes), f64(w.scale).astype(np.float32))


SHAPES = [(16, 16), (128, 256), (272, 144), (528, 1040), (1024, 2048)]


def _linear(dev, M, o, i, both=True):
    w, W = _weight(o, i, o + i, dev)
    x, dy = outliers((M, i), M).to(dev), normal((M, o), M + 1).to(dev)
    xq, dq = api.fp8_quantize_rows(x), api.fp8_quantize_rows(dy)
    X = blocks.row_values(f64(xq.codes), f64(xq.scale).astype(np.float32))
    dY = blocks.row_values(f64(dq.codes), f64(dq.scale).astype(np.float32))
    Y, dX = api.fp8_linear_fwd(w, xq), api.fp8_linear_bwd(w, dq)
    assert_product(f64(Y), X, W.T, "Y")
    assert_product(f64(dX), dY, W, "dX")
    if both:      # bf16 rows are quantized to the same codes, with the same sums
        assert torch.equal(api.fp8_linear_fwd(w, x), Y)
        assert torch.equal(api.fp8_linear_bwd(w, dy), dX)


@pytest.mark.parametrize("o,i", SHAPES)
@pytest.mark.parametrize("M", [1, 2, 8, 9, 16, 17, 33, 64, 77, 128, 129, 300])
def test_linear_fwd_bwd(cuda_device, M, o, i):
    _linear(cuda_device, M, o, i)


@pytest.mark.parametrize("M,o,i", [(700, 1024, 784), (1111, 528, 4096), (2048, 2064, 512)])
def test_linear_larger(cuda_device, M, o, i):
    _linear(cuda_device, M, o, i)


@pytest.mark.parametrize("M", [1, 8, 9, 16])
@pytest.mark.parametrize("o,i", [(2384, 2064), (4816, 1040)])
def test_linear_few_rows(cuda_device, M, o, i):
    """More blocks of 16 weight rows than SMs, and than SMs hold at once."""
    _linear(cuda_device, M, o, i)


@pytest.mark.parametrize("M", [17, 100, 130, 500])
@pytest.mark.parametrize("o,i", [(144, 4112), (4112, 144), (1040, 2048), (16, 11008), (2176, 2560)])
def test_linear_split_over_k(cuda_device, M, o, i):
    """Few tiles of a long K: 2, 4 or 8 CTAs share a tile's K, the last of them with fewer steps or none."""
    _linear(cuda_device, M, o, i)


@pytest.mark.parametrize("tile", ["128", "256", "pair"])
@pytest.mark.parametrize("M,o,i", [(1, 16, 16), (9, 272, 144), (129, 528, 1040), (300, 1024, 2048), (2048, 2064, 512)])
def test_linear_every_tile(cuda_device, monkeypatch, tile, M, o, i):
    monkeypatch.setenv("QLORA_B200_EXPERT_TILE", tile)
    _linear(cuda_device, M, o, i, both=False)


@pytest.mark.parametrize("M", [5, 300])
def test_nan_rows_stay_in_their_rows(cuda_device, M):
    w, W = _weight(272, 400, 2, cuda_device)
    x = normal((M, 400), 4)
    x[3, 140] = float("nan")
    Y = f64(api.fp8_linear_fwd(w, x.to(cuda_device)))
    assert np.isnan(Y[3]).all()
    keep = np.arange(M) != 3
    q, s = blocks.quantize_rows(f64(x)[keep])
    assert_product(Y[keep], blocks.row_values(q, s), W.T, "Y")
