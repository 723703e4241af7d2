"""GPU parity: linears grouped by expert (forward, dX, dW) in bf16 and e4m3 against fp64."""
import numpy as np
import pytest
import torch

from oracle import blocks
from quantized_lora_fine_b200 import api
from tests.block_helpers import assert_product, f64, normal, offsets_of, outliers

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status(cuda_device):
    yield
    torch.cuda.synchronize()
    assert api.status() == 0


GROUPS = {
    "one": [5],
    "single rows": [1, 1, 1, 1, 1],
    "with empty": [0, 3, 0, 0, 130, 1, 0],
    "all empty but one": [0, 0, 64, 0],
    "tile edges": [127, 128, 129, 255, 256, 257],
    "step edges": [63, 64, 65, 15, 16, 17, 33],
    "large": [700, 0, 1, 300],
}
SHAPES = [(16, 16), (144, 272), (528, 400), (256, 1024)]


def _run(dev, sizes, o, i, kind, before=0, after=0, seed=0):
    E = len(sizes)
    off = offsets_of(sizes, before)
    M = max(off[-1] + after, 1)
    X, dY = outliers((M, i), seed + 1), normal((M, o), seed + 2)
    W = normal((E, o, i), seed + 3, 0.05)
    for t in (X, dY):      # rows of no group hold what would spoil any sum they entered
        t[:before] = float("nan")
        t[off[-1]:] = float("nan")
    Xd, dYd, offs = X.to(dev), dY.to(dev), torch.tensor(off, dtype=torch.int32, device=dev)
    Y = torch.full((M, o), 7.0, dtype=torch.bfloat16, device=dev)
    dX = torch.full((M, i), 7.0, dtype=torch.bfloat16, device=dev)
    if kind == "fp8":
        w = api.fp8_quantize_weight(W.to(dev))
        Ws = [blocks.weight_values(f64(w.codes[e]), f64(w.scale[e]).astype(np.float32)) for e in range(E)]
        xq, dq = api.fp8_quantize_rows(Xd), api.fp8_quantize_rows(dYd)
        Xr = blocks.row_values(f64(xq.codes), f64(xq.scale).astype(np.float32))
        dYr = blocks.row_values(f64(dq.codes), f64(dq.scale).astype(np.float32))
        api.grouped_linear_fwd(w, Xd, offs, Y=Y)
        api.grouped_linear_bwd(w, None, dYd, offs, need_dW=False, dX=dX)
        dW = None
    else:
        w, Ws, Xr, dYr = W.to(dev), [f64(W[e]) for e in range(E)], f64(X), f64(dY)
        api.grouped_linear_fwd(w, Xd, offs, Y=Y)
        dW = torch.full((E, o, i), float("nan"), device=dev)
        api.grouped_linear_bwd(w, Xd, dYd, offs, dX=dX, dW=dW)
    Y, dX = f64(Y), f64(dX)
    for e, (a, b) in enumerate(blocks.spans(off)):
        assert_product(Y[a:b], Xr[a:b], Ws[e].T, f"Y of expert {e}")
        assert_product(dX[a:b], dYr[a:b], Ws[e], f"dX of expert {e}")
        if dW is not None:
            assert_product(f64(dW[e]), dYr[a:b].T, Xr[a:b], f"dW of expert {e}", bf16_out=False)
    for t in (Y, dX):
        assert (t[:before] == 7).all() and (t[off[-1]:] == 7).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("o,i", SHAPES)
@pytest.mark.parametrize("groups", list(GROUPS))
def test_grouped(cuda_device, groups, o, i, kind):
    _run(cuda_device, GROUPS[groups], o, i, kind)


@pytest.mark.parametrize("tile", ["128", "256", "pair"])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("o,i", [(144, 272), (528, 1024)])
@pytest.mark.parametrize("groups", list(GROUPS))
def test_grouped_every_tile(cuda_device, monkeypatch, tile, groups, o, i, kind):
    monkeypatch.setenv("QLORA_B200_EXPERT_TILE", tile)
    _run(cuda_device, GROUPS[groups], o, i, kind, before=1, after=30)


@pytest.mark.parametrize("sizes", [[1], [2, 1, 0, 3, 1, 1, 0, 1], [0, 0, 0, 9]])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_few_rows_a_group(cuda_device, sizes, kind):
    """The decoding kernel, with more rows in one group than it takes in a pass."""
    _run(cuda_device, sizes, 272, 1360, kind, before=0, after=0)


@pytest.mark.parametrize("o", [32, 1360, 2576])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_few_rows_of_few_and_many_ctas(cuda_device, o, kind):
    """16, 680 and 1288 blocks of 16 weight rows: each has its number of warps."""
    _run(cuda_device, [2, 1, 0, 18, 1, 1, 0, 9], o, 1104, kind)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("sizes", [[30, 0, 130], [0, 0, 40], [200], [1, 33, 15, 0, 40]])
@pytest.mark.parametrize("o,i", [(144, 4112), (2576, 272)])
def test_split_over_k(cuda_device, sizes, o, i, kind):
    """Few tiles of a long K, some clusters without a tile."""
    _run(cuda_device, sizes, o, i, kind, before=2, after=3)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("groups", ["with empty", "step edges", "large"])
def test_rows_outside_groups(cuda_device, groups, kind):
    """Rows before the first and behind the last group are neither read into a sum nor written."""
    _run(cuda_device, GROUPS[groups], 272, 144, kind, before=3, after=200)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_many_experts(cuda_device, kind):
    rng = np.random.default_rng(0)
    _run(cuda_device, list(rng.integers(0, 4, 1024)), 64, 48, kind)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_nan_of_one_expert_stays_there(cuda_device, kind):
    """Neighbouring experts' rows and weights share tiles and steps; a NaN in one reaches no other."""
    sizes, o, i = [70, 5, 90], 144, 208
    off = offsets_of(sizes)
    X, dY, W = normal((165, i), 1), normal((165, o), 2), normal((3, o, i), 3, 0.05)
    offs = torch.tensor(off, dtype=torch.int32, device=cuda_device)

    def run(X, dY, W):
        X, dY, W = X.to(cuda_device), dY.to(cuda_device), W.to(cuda_device)
        if kind == "fp8":
            w = api.fp8_quantize_weight(W)
            api.reset_status(api.Workspace.status_word(0))
            return (api.grouped_linear_fwd(w, X, offs), *api.grouped_linear_bwd(w, None, dY, offs, need_dW=False))
        return (api.grouped_linear_fwd(W, X, offs), *api.grouped_linear_bwd(W, X, dY, offs))

    clean = run(X, dY, W)
    X[70:75], dY[70:75], W[1] = float("nan"), float("inf"), float("nan")
    Y, dX, dW = run(X, dY, W)
    for rows in (slice(0, 70), slice(75, 165)):
        assert torch.equal(Y[rows], clean[0][rows]) and torch.equal(dX[rows], clean[1][rows])
    if kind == "bf16":
        assert torch.equal(dW[[0, 2]], clean[2][[0, 2]])


@pytest.mark.parametrize("M", [1000, 16384])
def test_dw_over_many_rows(cuda_device, M):
    """dW is summed in fp32 in spans of 256 rows: within a span the tensor cores make 16 additions that may cut off
    up to a whole last place (2^-23) of the partial sum, so a span is off by at most 16 2^-23 of its norm and spans of
    independent errors together by no more; the additions of the spans round, by 2^-24 each of a growing sum."""
    X, dY = normal((M, 256), 1).to(cuda_device), normal((M, 192), 2).to(cuda_device)
    W = torch.zeros((1, 192, 256), dtype=torch.bfloat16, device=cuda_device)
    offs = torch.tensor([0, M], dtype=torch.int32, device=cuda_device)
    _, dW = api.grouped_linear_bwd(W, X, dY, offs, need_dX=False)
    ref = f64(dY).T @ f64(X)
    assert np.linalg.norm(f64(dW[0]) - ref) <= 16 * 2.0 ** -23 * np.linalg.norm(ref)


def test_no_rows_at_all(cuda_device):
    """Every group empty: nothing is written but dW, which is zero."""
    X, dY, W = (normal(s, 1).to(cuda_device) for s in ((4, 32), (4, 48), (3, 48, 32)))
    offs = torch.full((4,), 2, dtype=torch.int32, device=cuda_device)
    Y = torch.full((4, 48), 7.0, dtype=torch.bfloat16, device=cuda_device)
    api.grouped_linear_fwd(W, X, offs, Y=Y)
    dX = torch.full((4, 32), 7.0, dtype=torch.bfloat16, device=cuda_device)
    _, dW = api.grouped_linear_bwd(W, X, dY, offs, dX=dX)
    assert (Y == 7).all() and (dX == 7).all() and not dW.any()


@pytest.mark.parametrize("off", [[0, 9, 4, 12], [-3, 5, 8, 12], [0, 5, 8, 99]])
def test_bad_offsets_are_reported(cuda_device, off):
    """Offsets that descend or leave the rows are clamped in the kernel and reported."""
    X, W = normal((12, 64), 1).to(cuda_device), normal((3, 32, 64), 2).to(cuda_device)
    offs = torch.tensor(off, dtype=torch.int32, device=cuda_device)
    Y = api.grouped_linear_fwd(W, X, offs)
    assert api.status() == 2          # QLORA_ERR_SHAPE
    api.reset_status(api.Workspace.status_word(0))
    run, want = 0, []
    for v in off:
        run = max(run, min(max(v, 0), 12))
        want.append(run)
    for e, (a, b) in enumerate(blocks.spans(want)):
        assert_product(f64(Y[a:b]), f64(X[a:b]), f64(W[e]).T, f"Y of expert {e}")


def test_one_expert_of_a_2d_weight(cuda_device):
    X, W = normal((77, 64), 1).to(cuda_device), normal((48, 64), 2).to(cuda_device)
    offs = torch.tensor([0, 77], dtype=torch.int32, device=cuda_device)
    assert_product(f64(api.grouped_linear_fwd(W, X, offs)), f64(X), f64(W).T, "Y")


def test_refused_calls(cuda_device):
    """What the binding refuses in words: shapes, types, kinds that do not go together, overlapping outputs."""
    W, X = normal((2, 64, 64), 1).to(cuda_device), normal((5, 64), 2).to(cuda_device)
    offs = torch.tensor([0, 2, 5], dtype=torch.int32, device=cuda_device)
    w8, x8 = api.fp8_quantize_weight(W), api.fp8_quantize_rows(X)
    bad = [
        (lambda: api.grouped_linear_fwd(W, x8, offs), "FP8Weight"),
        (lambda: api.grouped_linear_fwd(W, X[:, :32].contiguous(), offs), "columns"),
        (lambda: api.grouped_linear_fwd(W, X, offs.long()), "int32"),
        (lambda: api.grouped_linear_fwd(W, X, offs[:2]), "shape"),
        (lambda: api.grouped_linear_fwd(W, X, offs.cpu()), "CUDA"),
        (lambda: api.grouped_linear_fwd(W, X.float(), offs), "bfloat16"),
        (lambda: api.grouped_linear_fwd(W, X.t().contiguous().t(), offs), "contiguous"),
        (lambda: api.grouped_linear_fwd(W, X, offs, Y=X), "overlap"),
        (lambda: api.grouped_linear_bwd(W, X, X, offs, dX=X), "overlap"),
        (lambda: api.grouped_linear_bwd(W, X, X, offs, need_dX=False, need_dW=False), "must be true"),
        (lambda: api.grouped_linear_bwd(W, None, X, offs), "X is needed"),
        (lambda: api.grouped_linear_bwd(w8, X, X, offs), "frozen"),
        (lambda: api.fp8_linear_fwd(w8, X), "FP8Weight"),
        (lambda: api.FP8Rows(x8.codes, x8.scale[:4].contiguous()), "shape"),
        (lambda: api.FP8Weight(w8.codes, w8.scale[0]), "shape"),
    ]
    for call, words in bad:
        with pytest.raises(ValueError, match=words):
            call()
    with pytest.raises(RuntimeError, match="QLORA_ERR_SHAPE"):      # 40 is no multiple of 16
        api.grouped_linear_fwd(normal((2, 64, 40), 1).to(cuda_device), normal((5, 40), 2).to(cuda_device), offs)
    with pytest.raises(RuntimeError, match="QLORA_ERR_SHAPE"):      # no rows
        api.grouped_linear_fwd(W, X[:0], offs)
    with pytest.raises(RuntimeError, match="QLORA_ERR_ALIGN"):
        api.grouped_linear_fwd(W, normal((5 * 64 + 1,), 3).to(cuda_device)[1:].view(5, 64), offs)


def test_rows_and_scales_at_any_start(cuda_device):
    """Slices of larger tensors: rows from an odd one on, scales that start on no 16 bytes."""
    x = api.fp8_quantize_rows(normal((40, 640), 1).to(cuda_device))
    w = api.fp8_quantize_weight(normal((64, 640), 2, 0.05).to(cuda_device))
    W = blocks.weight_values(f64(w.codes), f64(w.scale).astype(np.float32))
    for first in (1, 3, 20):
        q = api.FP8Rows(x.codes[first:], x.scale[first:])
        X = blocks.row_values(f64(q.codes), f64(q.scale).astype(np.float32))
        assert_product(f64(api.fp8_linear_fwd(w, q)), X, W.T, "Y")
