"""The decoding kernel of the grouped linears: rows that all go to one expert, group tables longer than a warp."""
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


def _sizes(kind, E, M):
    n = [0] * E
    if kind == "first":
        n[0] = M
    elif kind == "last":
        n[-1] = M
    elif kind == "two":
        n[E // 3], n[E - 2] = M // 2, M - M // 2
    else:                     # a few groups of many passes among groups of one row and none
        rng = np.random.default_rng(E)
        for e in rng.integers(0, E, M // 2):
            n[e] += 1
        n[E // 2] += M - M // 2
    return n


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("kind", ["first", "last", "two", "mixed"])
@pytest.mark.parametrize("E", [2, 31, 32, 33, 70, 257, 1024])
def test_uneven_routing(cuda_device, E, kind, fmt):
    o, i = 48, 144
    sizes = _sizes(kind, E, 4 * E - 3)
    off = offsets_of(sizes, 2)
    M = off[-1] + 1
    X, W = outliers((M, i), E), normal((E, o, i), E + 1, 0.05)
    X[:2], X[-1:] = float("nan"), float("nan")
    offs = torch.tensor(off, dtype=torch.int32, device=cuda_device)
    Y = torch.full((M, o), 7.0, dtype=torch.bfloat16, device=cuda_device)
    if fmt == "fp8":
        w, x = api.fp8_quantize_weight(W.to(cuda_device)), api.fp8_quantize_rows(X.to(cuda_device))
        Xr = blocks.row_values(f64(x.codes), f64(x.scale).astype(np.float32))
        ws = lambda e: blocks.weight_values(f64(w.codes[e]), f64(w.scale[e]).astype(np.float32))
    else:
        w, x, Xr, ws = W.to(cuda_device), X.to(cuda_device), f64(X), lambda e: f64(W[e])
    api.grouped_linear_fwd(w, x, offs, Y=Y)
    Y = f64(Y)
    for e, (a, b) in enumerate(blocks.spans(off)):
        if b > a:
            assert_product(Y[a:b], Xr[a:b], ws(e).T, f"Y of expert {e}")
    assert (Y[:2] == 7).all() and (Y[-1:] == 7).all()


@pytest.mark.parametrize("E", [32, 70])
@pytest.mark.parametrize("at,value", [(0, -4), (1, 100000), (31, 3), (-2, -1), (-1, 100000)])
def test_bad_offsets_of_many_groups(cuda_device, E, at, value):
    """Taken as the running maximum of the clamped values, and reported."""
    sizes = [2] * E
    off = offsets_of(sizes)
    M = off[-1]
    off[at] = value
    X, W = normal((M, 64), 1), normal((E, 32, 64), 2)
    offs = torch.tensor(off, dtype=torch.int32, device=cuda_device)
    Y = f64(api.grouped_linear_fwd(W.to(cuda_device), X.to(cuda_device), offs))
    assert api.status() == 2          # QLORA_ERR_SHAPE
    api.reset_status(api.Workspace.status_word(0))
    run, want = 0, []
    for v in off:
        run = max(run, min(max(v, 0), M))
        want.append(run)
    for e, (a, b) in enumerate(blocks.spans(want)):
        if b > a:
            assert_product(Y[a:b], f64(X[a:b]), f64(W[e]).T, f"Y of expert {e}")


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_one_group_with_every_row_takes_no_longer_than_even_groups(cuda_device, fmt):
    """4096 rows over 1024 experts: evenly, every weight is read once (134 MB in bf16); with all rows in one group no
    more than that group's is needed. One CTA for all of a group's passes took many times the even time here."""
    E, o, i = 1024, 256, 256
    W = normal((E, o, i), 1, 0.05).to(cuda_device)
    x = normal((4 * E, i), 2).to(cuda_device)
    if fmt == "fp8":
        W, x = api.fp8_quantize_weight(W), api.fp8_quantize_rows(x)
    Y = torch.empty((4 * E, o), dtype=torch.bfloat16, device=cuda_device)

    def time(sizes):
        offs = torch.tensor(offsets_of(sizes), dtype=torch.int32, device=cuda_device)
        best = float("inf")
        for _ in range(10):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            a.record()
            for _ in range(5):
                api.grouped_linear_fwd(W, x, offs, Y=Y)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    assert time([4 * E] + [0] * (E - 1)) <= 2 * time([4] * E)
