"""The norm, the 8-bit linear and the grouped linears used together, captured, on several streams, and at
sizes past 32-bit offsets."""
import numpy as np
import pytest
import torch

from oracle import blocks
from quantized_lora_fine_b200 import api
from tests.block_helpers import U_BF16, assert_product, bf16_round, f64, normal, offsets_of, outliers

pytestmark = pytest.mark.gpu

EPS = 1e-6
H, F, E = 512, 272, 4
SIZES = [37, 0, 90, 6]


@pytest.fixture(autouse=True)
def _clean_status(cuda_device):
    yield
    torch.cuda.synchronize()
    assert api.status() == 0


def _block_inputs(dev, seed=0):
    M = sum(SIZES)
    d = dict(x=outliers((M, H), seed), r=normal((M, H), seed + 1), w=(1 + 0.1 * normal((H,), seed + 2).float()),
             up=normal((H, H), seed + 3, 0.04), experts=normal((E, F, H), seed + 4, 0.04), g=normal((M, F), seed + 5))
    d["w"] = d["w"].to(torch.bfloat16)
    d = {k: v.to(dev) for k, v in d.items()}
    d["off"] = torch.tensor(offsets_of(SIZES), dtype=torch.int32, device=dev)
    d["up8"] = api.fp8_quantize_weight(d["up"])
    return d


def _block(d):
    """norm -> 8-bit linear -> experts, and the gradients back to the block's input."""
    q, h, rstd = api.rms_norm_fwd(d["x"], d["w"], EPS, residual=d["r"], fp8=True)
    z = api.fp8_linear_fwd(d["up8"], q)
    y = api.grouped_linear_fwd(d["experts"], z, d["off"])
    dz, dW = api.grouped_linear_bwd(d["experts"], z, d["g"], d["off"])
    dn = api.fp8_linear_bwd(d["up8"], dz)
    dx, dw = api.rms_norm_bwd(dn, h, rstd, d["w"])
    return dict(codes=q.codes, scale=q.scale, h=h, rstd=rstd, z=z, y=y, dz=dz, dW=dW, dn=dn, dx=dx, dw=dw)


def test_block_forward_and_backward(cuda_device):
    """Every stage against fp64 on the values that reached it, and the whole gradient against the chain
    in fp64."""
    d = _block_inputs(cuda_device)
    o = {k: f64(v) for k, v in _block(d).items()}
    assert np.array_equal(o["h"], bf16_round(f64(d["x"]) + f64(d["r"])))
    W8 = blocks.weight_values(f64(d["up8"].codes), f64(d["up8"].scale).astype(np.float32))
    X8 = blocks.row_values(o["codes"], o["scale"].astype(np.float32))
    assert_product(o["z"], X8, W8.T, "z")
    off = offsets_of(SIZES)
    Ws = [f64(d["experts"][e]) for e in range(E)]
    for e, (a, b) in enumerate(blocks.spans(off)):
        assert_product(o["y"][a:b], o["z"][a:b], Ws[e].T, "y")
        assert_product(o["dz"][a:b], f64(d["g"])[a:b], Ws[e], "dz")
        assert_product(o["dW"][e], f64(d["g"])[a:b].T, o["z"][a:b], "dW", bf16_out=False)
    q, s = blocks.quantize_rows(o["dz"])
    assert_product(o["dn"], blocks.row_values(q, s), W8, "dn")
    # the chain without any rounding of the gradients: e4m3 rounds dz by at most 2^-4 of each value (2^-4 / 448 of
    # its block's largest below the normal range), which reaches dx through |W8| and the norm
    dz = np.concatenate([f64(d["g"])[a:b] @ Ws[e] for e, (a, b) in enumerate(blocks.spans(off))])
    dn = dz @ W8
    dx, _ = blocks.rms_norm_backward(dn, o["h"], f64(d["w"]), EPS)
    big = np.repeat(np.abs(dz).reshape(len(dz), -1, 128).max(2), 128, 1)
    err = (np.abs(dz) * (2.0 ** -4 + 2 * U_BF16) + big * 2.0 ** -10 / 448) @ np.abs(W8) * (1 + U_BF16) + U_BF16 * np.abs(dn)
    _, rstd = blocks.rms_norm(o["h"], f64(d["w"]), EPS)
    n, w = np.abs(o["h"]) * rstd[:, None], np.abs(f64(d["w"]))
    bound = rstd[:, None] * (err * w + n * (err * w * n).mean(1, keepdims=True))
    assert np.all(np.abs(o["dx"] - dx) <= bound * 1.01 + 2 * U_BF16 * np.abs(dx) + 1e-4 * bound.max())


def test_nf4_experts(cuda_device):
    """Experts kept in NF4 as one stacked weight, decoded for the grouped products."""
    Wt = normal((E * F, H), 3, 0.04).to(cuda_device)
    W = api.dequantize(api.quantize(Wt, double_quant=True)).view(E, F, H)
    X = normal((sum(SIZES), H), 1).to(cuda_device)
    off = offsets_of(SIZES)
    Y = api.grouped_linear_fwd(W, X, torch.tensor(off, dtype=torch.int32, device=cuda_device))
    for e, (a, b) in enumerate(blocks.spans(off)):
        assert_product(f64(Y[a:b]), f64(X[a:b]), f64(W[e]).T, "Y")


def test_captured_and_replayed(cuda_device):
    """A graph of the block gives the eager call's bits, also on new inputs copied into its own; two graphs
    replayed at once on two streams do not disturb each other."""
    ins = [_block_inputs(cuda_device, s) for s in (0, 100)]
    want = [_block(d) for d in ins]
    graphs, outs = [], []
    for d in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_block(d))
        graphs.append(g)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        for st, g in zip((s1, s2), graphs):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            for k in w:
                assert torch.equal(w[k], o[k]), k
    # new inputs in the first graph's tensors
    new = _block_inputs(cuda_device, 200)
    for k in ("x", "r", "g"):
        ins[0][k].copy_(new[k])
    new.update(w=ins[0]["w"], up8=ins[0]["up8"], experts=ins[0]["experts"])
    ref = _block(new)
    graphs[0].replay()
    torch.cuda.synchronize()
    for k in ref:
        assert torch.equal(ref[k], outs[0][k]), k


def test_two_streams_at_once(cuda_device):
    ins = [_block_inputs(cuda_device, s) for s in (0, 100)]
    want = [_block(d) for d in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        got = []
        for d, st in zip(ins, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(_block(d))
        torch.cuda.synchronize()
        for w, o in zip(want, got):
            for k in w:
                assert torch.equal(w[k], o[k]), k


def test_back_to_back_calls_do_not_overtake(cuda_device):
    """Each kernel may start while the one before it ends: a chain that feeds every output on, many times."""
    w = api.fp8_quantize_weight(normal((512, 512), 1, 0.06).to(cuda_device))
    one = torch.ones(512, dtype=torch.bfloat16, device=cuda_device)

    def chain(sync):
        x = normal((300, 512), 2).to(cuda_device)
        for _ in range(20):
            q, _, _ = api.rms_norm_fwd(x, one, EPS, fp8=True)
            x = api.fp8_linear_fwd(w, q)
            if sync:
                torch.cuda.synchronize()
        return x

    assert torch.equal(chain(False), chain(True))


@pytest.mark.parametrize("M", [1, 12, 300])
def test_operands_written_by_the_call_before(cuda_device, M):
    """Weights, scales, rows and norm weights that the call before writes, into memory that held others: as with
    a wait after every call."""
    Ws = [normal((2, 512, 512), i, 0.06).to(cuda_device) for i in range(6)]
    off = torch.tensor([0, M // 3, M], dtype=torch.int32, device=cuda_device)
    api.fp8_quantize_weight(Ws[0])

    def chain(sync):
        wait = torch.cuda.synchronize if sync else (lambda: None)
        x = normal((M, 512), 9).to(cuda_device)
        for W in Ws:
            w = api.fp8_quantize_weight(W[0])
            wait()
            x = api.fp8_linear_fwd(w, x)
            wait()
            w = api.fp8_quantize_weight(W)
            wait()
            y = api.grouped_linear_fwd(w, x, off)
            wait()
            _, _, rstd = api.rms_norm_fwd(x, W[0, 0], EPS)
            wait()
            _, dw = api.rms_norm_bwd(y, x, rstd, W[0, 0])
            wait()
            x, _, _ = api.rms_norm_fwd(y, dw, EPS, residual=x)
            wait()
        return x

    x = chain(True)
    assert x.isfinite().all() and torch.equal(chain(False), x)


def test_offsets_past_32_bits(cuda_device):
    """Rows, weights and outputs whose byte or element offsets pass 2^32."""
    dev = cuda_device
    n = 4096
    M = (1 << 20) + 65                       # M n > 2^32 bf16 values
    x = torch.empty((M, n), dtype=torch.bfloat16, device=dev)
    tail = normal((130, n), 5)
    x[-130:] = tail.to(dev)
    x[:-130] = 0
    q = api.fp8_quantize_rows(x)
    codes, scale = blocks.quantize_rows(f64(tail))
    assert np.array_equal(f64(q.codes[-130:]), codes) and np.array_equal(f64(q.scale[-130:]), scale)
    y, _, rstd = api.rms_norm_fwd(x, torch.ones(n, dtype=torch.bfloat16, device=dev), EPS)
    yr, _ = blocks.rms_norm(f64(tail), np.ones(n), EPS)
    assert np.all(np.abs(f64(y[-130:]) - yr) <= (U_BF16 + 2.0 ** -12) * np.abs(yr) + 2.0 ** -134)
    del x, y
    w = api.fp8_quantize_weight(normal((n, n), 6, 0.02).to(dev))
    Y = api.fp8_linear_fwd(w, q)
    assert_product(f64(Y[-130:, :64]), blocks.row_values(codes, scale),
                   blocks.weight_values(f64(w.codes), f64(w.scale).astype(np.float32))[:64].T, "Y")
    del q, Y
    torch.cuda.empty_cache()
    E2, o, i = 80, 8192, 8192                # 5.4e9 weights
    W = torch.zeros((E2, o, i), dtype=torch.bfloat16, device=dev)
    last = normal((o, i), 7, 0.02)
    W[-1] = last.to(dev)
    for sizes in ([0] * (E2 - 1) + [150], [0] * (E2 - 1) + [3]):
        X = normal((sizes[-1], i), 8)
        offs = torch.tensor(offsets_of(sizes), dtype=torch.int32, device=dev)
        Y = api.grouped_linear_fwd(W, X.to(dev), offs)
        assert_product(f64(Y[:, -64:]), f64(X), f64(last[-64:]).T, "Y of the last expert")
        dX, _ = api.grouped_linear_bwd(W, None, X.to(dev), offs, need_dW=False)
        assert_product(f64(dX[:, -64:]), f64(X), f64(last[:, -64:]), "dX of the last expert")
    dW = torch.empty((E2, o, i), dtype=torch.float32, device=dev)
    api.grouped_linear_bwd(W, X.to(dev), X.to(dev), offs, need_dX=False, dW=dW)
    assert_product(f64(dW[-1, -64:, -64:]), f64(X)[:, -64:].T, f64(X)[:, -64:], "dW", bf16_out=False)
    assert not dW[:-1].any()
